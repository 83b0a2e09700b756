"""The 8-bit cache at the ends of its range: queries near the type's largest number."""
import pytest
import torch

from test_gpu_kv8 import decode_and_check, problem

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
