"""attn_kv4_decode where its powers of two end: values next to nothing under nearly all the weight, queries
near the type's largest number."""
import math

import pytest
import torch

import plain64
from plain64 import DT
from test_gpu_kv4_decode import decode_and_check, i32, problem, reference, wide

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


def heavy_token(d, dtype, gap, size, lens=(200, 700)):
    """Token 5 of the first request has a score 2^gap times the others' in weight and the value zero, as append writes
    it; the others' scales are `size` times a cache's usual ones."""
    q, kc, vc, ks, vs, table = problem(list(lens), 1, 4, 1, d, 16, dtype, seed=gap + d)
    q.fill_(0.25)
    ks.fill_(0.002)
    at = table[0, 0].item()
    kc[at, 0, 5], ks[at, 0, 5] = 0x77, gap * math.log(2) / (1.5 * d)    # all sixes: q k = 1.5 d ks
    vs *= size
    vc[at, 0, 5], vs[at, 0, 5] = 0, 2.0 ** -64
    return [q, kc, vc, ks, vs, table]


def check_both_ways(args, said, dtype):
    """Against the reference and bounds of `said`.  (The second request's outputs, of 2^40 and more, are infinite in fp16.)"""
    from exact_tiled_attention_22_gb300 import attn
    (ro, bo), (rl, bl) = reference(said, [200, 700], 1.0, True, dtype)
    ro = torch.where(ro.abs() > torch.finfo(DT[dtype]).max, ro * math.inf, ro)
    assert not torch.isinf(ro[0]).any()
    for table in (args[5], wide(args[5])):
        o, lse = attn.kv4_decode(*(x.cuda() for x in (*args[:-1], table)), i32([200, 700]), 1.0)
        plain64.check(lse, rl, bl, "lse")
        plain64.check(o, ro, bo, "o")
    assert o[0].abs().amax() > 0.25


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gap", [45, 50, 55, 60, 75])
def test_decode_a_heavy_token_whose_value_is_zero(d, dtype, gap):
    """Outputs of size one, all of them from tokens whose weights are 2^-gap: they keep their precision."""
    args = heavy_token(d, dtype, gap, 2.0 ** gap)
    check_both_ways(args, args, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_a_heavier_token_whose_value_is_zero(d, dtype):
    """A weight of 2^82 times the others': its zero counts as 2^-80 of the tile's largest scale, and the others'
    products are within 2^-21 or 2^-25 of that.  (Codes of zero: scales that say so change no value.)"""
    args = heavy_token(d, dtype, 82, 2.0 ** 82)
    said = [x.clone() for x in args]
    said[4][args[5][0, 0].item(), 0, 5] = 2.0 ** 82 * 2.0 ** -80
    check_both_ways(args, said, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [4, 8, 16])
def test_decode_queries_up_to_the_largest_number(d, Hq):
    """Elements up to bf16's largest, 2^128 less a step: no more than 2^-21 of the row's largest is lost."""
    g = torch.Generator().manual_seed(40)
    args = problem([300, 17], 1, Hq, 1, d, 16, "bf16", seed=41)
    top = torch.finfo(torch.bfloat16).max
    args[0].copy_((torch.rand(args[0].shape, generator=g, dtype=torch.float64) * 2 - 1) * top)
    args[0][:, :, ::2, 3] = top
    args[3].copy_(args[3] * 2.0 ** -60)
    decode_and_check(args, [300, 17], 2.0 ** -66, True, "bf16")
