"""attn_kv4_decode beside other kernels, and on each of the ways it takes through its tiles."""
import math
import random

import pytest
import torch

import plain64
from test_gpu_kv4_decode import i32, problem, reference, wide

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


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (64, "bf16"), (128, "bf16")])
def test_decodes_and_prompts_in_turn_on_two_streams(d, dtype):
    """Clusters, dealt tiles and packed prompts, one after the other on each of two streams: all of them take tensor
    memory, and the next one's blocks come while this one's are at work."""
    from exact_tiled_attention_22_gb300 import attn
    lens = [900, 17, 700]
    args = [x.cuda() for x in problem(lens, 1, 16, 4, d, 64, dtype, seed=30)]
    ln, narrow = i32(lens), args.pop()
    tables = (narrow, wide(narrow))
    g = torch.Generator().manual_seed(31)
    q = torch.randn((700, 8, d), generator=g).to(args[0].dtype).cuda()
    k, v = (torch.randn((700, 2, d), generator=g).to(args[0].dtype).cuda() for _ in range(2))
    cu = i32([0, 130, 700])

    def run():
        return [*attn.kv4_decode(*args, tables[0], ln), *attn.varlen_fwd(q, k, v, cu, cu, None, True),
                *attn.kv4_decode(*args, tables[0], ln), *attn.kv4_decode(*args, tables[1], ln),
                *attn.varlen_fwd(q, k, v, cu, cu, None, True)]

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(x, y) for x, y in zip(r, want))


def decode_by(args, table, lens, scale, ws=None):
    """(o, lse) and whether a merge kernel ran: the tiles were dealt to all blocks, and not to clusters."""
    from exact_tiled_attention_22_gb300 import attn
    attn.attn_profile_begin()
    o, lse = attn.kv4_decode(*(x.cuda() for x in (*args[:-1], table)), i32(lens), scale, ws=ws)
    ran = attn.attn_profile_end()
    attn.check(attn.attn_status())
    assert ran["attn_kv4_split"][0] == 1
    return o, lse, ran["attn_kv4_merge"][0] == 1


def spread(n, lo, hi, seed):
    rng = random.Random(seed)
    return [int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) for _ in range(n)]


DEALT = [
    # (lens, Hq, Hkv, d, page, dtype, whether there are units enough for shares of 8 and 7)
    ([17001, 9000, 2300, 130, 1, 0, 4000], 32, 8, 128, 64, "bf16", True),   # long segments cut between shares
    ([33001, 17000, 9001, 130, 1, 0, 4100], 32, 8, 64, 128, "bf16", True),
    (spread(40, 100, 3000, 1), 16, 8, 128, 64, "bf16", True),
    (spread(40, 200, 5000, 2), 8, 8, 64, 32, "bf16", True),
    (spread(150, 50, 1500, 3), 16, 4, 128, 64, "bf16", True),               # more requests than a warp deals
    (spread(150, 50, 2500, 4) + [0, 3], 16, 4, 64, 64, "bf16", True),
    ([0, 600, 1] + spread(140, 1, 600, 5), 16, 2, 128, 32, "bf16", False),  # ... with 8 rows, 16, and in fp16
    ([0, 600, 1] + spread(140, 1, 600, 6), 16, 2, 64, 16, "fp16", False),
    (spread(137, 1, 700, 7) + [0, 0], 32, 2, 128, 64, "bf16", False),
    (spread(137, 1, 700, 8) + [0, 0], 32, 2, 64, 32, "bf16", False),
    (spread(137, 1, 700, 9) + [0, 0], 8, 2, 128, 64, "fp16", False),
]


@pytest.mark.parametrize("case", DEALT, ids=lambda c: f"B{len(c[0])}h{c[1]}x{c[2]}d{c[3]}{c[5]}")
def test_dealt_tiles(case):
    """Also with a workspace full of NaN: parts lie where the merge looks for them, in unequal shares, too."""
    from exact_tiled_attention_22_gb300 import attn
    lens, Hq, H, d, page, dtype, weighted = case
    args = problem(lens, 1, Hq, H, d, page, dtype, seed=sum(lens))
    units = sum(-(-n // (128 * 128 // d)) + 1 for n in lens if n) * H
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (units >= 4 * 3 * sms and Hq // H <= 4 and dtype == "bf16") == weighted
    (ro, bo), (rl, bl) = reference(args, lens, d ** -0.5, True, dtype)
    dirty = torch.full((attn.attn_kv4_decode_workspace_size(1, Hq, H, d) // 4,), math.nan, device="cuda")
    o, lse, dealt = decode_by(args, wide(args[-1]), lens, d ** -0.5, dirty)
    assert dealt
    plain64.check(lse, rl, bl, "lse")
    plain64.check(o, ro, bo, "o")


CLUSTERS = [
    # (lens, Hq, Hkv, d, page, dtype)
    ([2100], 4, 1, 128, 16, "bf16"),            # a cluster of 16, 17 tiles
    ([4300, 0], 7, 1, 64, 64, "fp16"),          # ... of 8 rows
    ([2500, 1], 16, 1, 128, 128, "bf16"),       # ... of 16
    ([1300] * 12, 32, 8, 128, 64, "bf16"),      # of four
    ([700] * 8, 64, 8, 64, 32, "bf16"),         # of four, 8 rows
    ([511, 77, 0], 16, 1, 128, 16, "bf16"),
]


@pytest.mark.parametrize("case", CLUSTERS, ids=lambda c: f"B{len(c[0])}h{c[1]}x{c[2]}d{c[3]}{c[5]}")
def test_clusters(case):
    lens, Hq, H, d, page, dtype = case
    args = problem(lens, 1, Hq, H, d, page, dtype, seed=sum(lens))
    (ro, bo), (rl, bl) = reference(args, lens, d ** -0.5, True, dtype)
    for table, by_merge in ((args[-1], False), (wide(args[-1]), True)):
        o, lse, dealt = decode_by(args, table, lens, d ** -0.5)
        assert dealt == by_merge
        plain64.check(lse, rl, bl, "lse")
        plain64.check(o, ro, bo, "o")
