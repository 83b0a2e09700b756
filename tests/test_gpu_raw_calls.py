"""The packed and serving entry points that mirror the C ABI, on the caller's buffers and
stream: the bits of the conveniences."""
import pytest
import torch

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


def test_packed_calls():
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(1)
    Hq, H, d, Tq, Tk = 6, 2, 64, 300, 2400
    q, do = (torch.randn((Tq, Hq, d), generator=g).half().cuda() for _ in range(2))
    kv = torch.randn((Tk, 2 * H, d), generator=g).half().cuda()  # k and v beside one another
    k, v = kv[:, :H], kv[:, H:]
    cq, ck = i32([0, 200, 300]), i32([0, 1400, 2400])
    o, lse = torch.empty_like(q), torch.empty((Hq, Tq), device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty((Tk, H, d), dtype=q.dtype, device="cuda"), torch.empty((Tk, H, d), dtype=q.dtype, device="cuda")
    n = attn.attn_varlen_fwd_workspace_size(2, Tq, Tk, Hq, H, d)
    m = attn.attn_varlen_bwd_workspace_size(2, Tq, Hq, H, d)
    ws = torch.empty(max(n, m), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    attn.check(attn.attn_varlen_fwd(q, k, v, o, lse, cq, ck, 2, Tq, Tk, Hq, H, d, Hq * d, 2 * H * d, 2 * H * d, 0.1, True,
                                    "fp16", ws, n, side))
    attn.check(attn.attn_varlen_bwd(q, k, v, o, lse, do, dq, dk, dv, cq, ck, 2, Tq, Tk, Hq, H, d, Hq * d, 2 * H * d,
                                    2 * H * d, 0.1, True, "fp16", ws, m, side))
    side.synchronize()
    o2, lse2 = attn.varlen_fwd(q, k, v, cq, ck, 0.1, True)
    dq2, dk2, dv2 = attn.varlen_bwd(q, k, v, o2, lse2, do, cq, ck, 0.1, True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(dk, dk2) and torch.equal(dv, dv2)
    # |dQ|: fp32 sums of the same terms in another order, then one fp16 rounding each
    assert (dq.float() - dq2.float()).abs().max() <= 2.0 ** -10 * dq2.float().abs().max()


def test_a_decoding_step():
    from exact_tiled_attention_22_gb300 import attn
    g = torch.Generator().manual_seed(2)
    B, H, Hq, d, page, width, P = 5, 2, 8, 128, 16, 6, 40
    new = torch.randn((B, 2, H, d), generator=g).bfloat16().cuda()
    q = torch.randn((B, 1, Hq, d), generator=g).bfloat16().cuda()

    def state():
        gg = torch.Generator().manual_seed(3)
        table = torch.randperm(P, generator=gg)[:B * width].int().view(B, width).cuda()
        codes = [torch.randint(0, 120, (P, H, page, d), generator=gg, dtype=torch.uint8).cuda() for _ in range(2)]
        scales = [torch.full((P, H), 2.0 ** -6, device="cuda") for _ in range(2)]
        left = [p for p in range(P) if p not in table.flatten().tolist()]
        return i32([0, 15, 16, 33, 90]), table, i32(left + [-1] * 30), i32([len(left)]), codes, scales

    lens, table, stack, count, (kc, vc), (ks, vs) = state()
    cap = stack.numel()
    add, granted, cu, slots = i32([1] * B), i32([0] * B), i32([0] * (B + 1)), torch.empty(B, dtype=torch.int64, device="cuda")
    attn.check(attn.attn_pages_extend(lens, add, B, table, width, stack, count, cap, page, B, lens, granted, cu, slots, count))
    attn.check(attn.attn_kv8_append(new[:, 0], new[:, 1], 2 * H * d, 2 * H * d, slots, B, H, d, kc, vc, ks, vs, P, page,
                                    torch.bfloat16))
    o, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
    n = attn.attn_kv8_decode_workspace_size(1, Hq, H, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    attn.check(attn.attn_kv8_decode(q, kc, vc, ks, vs, table, lens, o, lse, B, 1, Hq, H, d, P, page, width, 0.1, True,
                                    "bf16", ws, n))
    done = i32([0, 1, 0, 1, 1])
    attn.check(attn.attn_pages_release(lens, done, B, table, width, stack, count, cap, page, lens, count))
    mine = (lens, table, stack, count, kc, vc, ks, vs, slots, cu, granted, o, lse)

    lens, table, stack, count, (kc, vc), (ks, vs) = state()
    _, granted, cu, slots, _ = attn.pages_extend(lens, add, table, stack, count, page, B, new_lens=lens, free_left=count)
    attn.kv8_append(new[:, 0], new[:, 1], slots, kc, vc, ks, vs)
    o, lse = attn.kv8_decode(q, kc, vc, ks, vs, table, lens, 0.1)
    attn.pages_release(lens, done, table, stack, count, page, new_lens=lens, free_left=count)
    for a, b in zip(mine, (lens, table, stack, count, kc, vc, ks, vs, slots, cu, granted, o, lse)):
        assert torch.equal(a, b)
    assert torch.isfinite(lse).all() and count.item() > 0
