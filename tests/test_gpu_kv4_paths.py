"""attn_kv4_decode beside other kernels, and on each of the ways it takes through its tiles."""
import pytest
import torch

from test_gpu_kv4_decode import i32, problem, wide

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
