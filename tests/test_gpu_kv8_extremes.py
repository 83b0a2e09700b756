"""The 8-bit cache at the ends of its range: queries near the type's largest number, scales of 24 bits."""
import numpy as np
import pytest
import torch

from plain64 import DT
from test_gpu_kv8 import F8, decode_and_check, problem

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [4, 8, 16])
def test_decode_queries_up_to_the_largest_number(d, Hq):
    """Elements up to bf16's largest, 2^128 less a step: no more than 2^-21 of the row's largest is lost."""
    g = torch.Generator().manual_seed(40)
    args = problem([300, 17], 1, Hq, 1, d, 16, "bf16", seed=41)
    top = torch.finfo(torch.bfloat16).max
    args[0].copy_((torch.rand(args[0].shape, generator=g, dtype=torch.float64) * 2 - 1) * top)
    args[0][:, :, ::2, 3] = top
    args[3].mul_(2.0 ** -60)
    decode_and_check(args, [300, 17], 2.0 ** -70, True, "bf16")


def nearest(x, dtype):
    """Float64 to the 16-bit type in one rounding, to nearest even, at most the type's largest."""
    x = x.clamp(-torch.finfo(DT[dtype]).max, torch.finfo(DT[dtype]).max)
    if dtype == "fp16":
        return torch.from_numpy(x.numpy().astype(np.float16))
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256), e - 8).bfloat16()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -20, 300.0])
def test_read_rounds_products_with_any_scale_once(dtype, size):
    """Products of a code (4 bits) and a scale (24 bits) have 28 bits: rounded to 32-bit numbers first, some of
    them would end on a border of the 16-bit type and go to the wrong side."""
    from exact_tiled_attention_22_gb300 import attn
    P, H, page, d = 6000, 4, 16, 64
    g = torch.Generator().manual_seed(50)
    codes = torch.randint(0, 256, (2, P, H, page, d), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x7E
    scales = (torch.rand((2, P, H), generator=g) + 0.5) * size
    want = [nearest((c.view(F8).double() * s.double()[..., None, None]).transpose(1, 2).reshape(-1, H, d), dtype)
            for c, s in zip(codes, scales)]
    twice = sum(((c.view(F8).float() * s[..., None, None]).clamp(-6e4, 6e4).transpose(1, 2).reshape(-1, H, d).to(DT[dtype]) !=
                 w.clamp(-6e4, 6e4)).sum().item() for c, s, w in zip(codes, scales, want))
    assert twice > 0                       # (there are such products among them)
    got = attn.kv8_read(codes[0].cuda().view(F8), codes[1].cuda().view(F8), scales[0].cuda(), scales[1].cuda(),
                        torch.arange(P, dtype=torch.int32)[None].cuda(), torch.tensor([P * page], dtype=torch.int32).cuda(),
                        torch.tensor([0, P * page], dtype=torch.int32).cuda(), P * page, DT[dtype])
    for x, w in zip(got, want):
        assert torch.equal(x.cpu().view(torch.int16), w.view(torch.int16))
