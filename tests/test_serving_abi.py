"""What the packed and paged calls refuse on the host, before any device work
(no GPU needed), and their workspace sizes."""
import pytest
import torch


@pytest.fixture(scope="module")
def A():
    from exact_tiled_attention_22_gb300 import build
    build.build()
    from exact_tiled_attention_22_gb300 import attn
    return attn


# Fake aligned addresses, far apart: every call below is refused on the host.
P = [0x100000000 * (i + 1) for i in range(20)]
WS = 1 << 44


def call(fn, names, base, **kw):
    args = dict(base)
    unknown = set(kw) - set(args)
    assert not unknown, unknown
    args.update(kw)
    return fn(*(args[n] for n in names.split()))


EXTEND = "lens add B table width free count cap page T new_lens granted cu slots left stream"


def extend(A, **kw):
    base = dict(lens=P[0], add=P[1], B=4, table=P[2], width=8, free=P[3], count=P[4], cap=100, page=16, T=10,
                new_lens=P[5], granted=P[6], cu=P[7], slots=P[8], left=P[9], stream=None)
    return call(A.lib.attn_pages_extend, EXTEND, base, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), -1), (dict(free=None), -1), (dict(left=None), -1), (dict(slots=None), -1), (dict(B=0), -1),
    (dict(width=0), -1), (dict(cap=0), -1), (dict(B=8193), -2), (dict(page=8), -2), (dict(page=48), -2),
    (dict(page=256), -2), (dict(T=-1), -1), (dict(T=1 << 31), -1), (dict(width=1 << 27), -1),
    (dict(add=P[1] + 2), -3), (dict(slots=P[8] + 4), -3),
    (dict(granted=P[1]), -1), (dict(table=P[0]), -1), (dict(new_lens=P[0] + 4), -1), (dict(cu=P[6]), -1),
    (dict(left=P[0]), -1), (dict(slots=P[3]), -1)])
def test_extend_refuses(A, kw, code):
    assert extend(A, **kw) == code and A.last_error()


RELEASE = "lens done B table width free count cap page new_lens left stream"


@pytest.mark.parametrize("kw,code", [
    (dict(done=None), -1), (dict(B=0), -1), (dict(page=1), -2), (dict(free=P[3] + 1), -3), (dict(free=P[2]), -1),
    (dict(left=P[3]), -1), (dict(new_lens=P[1]), -1)])
def test_release_refuses(A, kw, code):
    base = dict(lens=P[0], done=P[1], B=4, table=P[2], width=8, free=P[3], count=P[4], cap=100, page=16,
                new_lens=P[5], left=P[6], stream=None)
    assert call(A.lib.attn_pages_release, RELEASE, base, **kw) == code


APPEND = "k v ks vs slots T H d kc vc sk sv P page dtype stream"


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(sv=None), -1), (dict(T=-1), -1), (dict(H=0), -1), (dict(P=0), -1), (dict(d=96), -2),
    (dict(dtype=3), -2), (dict(page=24), -2), (dict(T=1 << 30), -1), (dict(P=1 << 30, H=2), -1),
    (dict(ks=120), -1), (dict(vs=132), -1), (dict(k=P[0] + 8), -3), (dict(kc=P[3] + 4), -3), (dict(sk=P[5] + 2), -3),
    (dict(slots=P[2] + 4), -3), (dict(kc=P[0]), -1), (dict(vc=P[3]), -1), (dict(sk=P[2]), -1)])
def test_append_refuses(A, kw, code):
    base = dict(k=P[0], v=P[1], ks=128, vs=128, slots=P[2], T=5, H=2, d=64, kc=P[3], vc=P[4], sk=P[5], sv=P[6], P=9,
                page=16, dtype=A.ATTN_F16, stream=None)
    assert call(A.lib.attn_kv8_append, APPEND, base, **kw) == code and A.last_error()


DECODE = "q kc vc sk sv table lens o lse B Nq Hq H d P page width scale causal dtype ws ws_bytes stream"


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(table=None), -1), (dict(B=0), -1), (dict(Nq=0), -1), (dict(Hq=3), -1), (dict(H=0), -1),
    (dict(d=32), -2), (dict(dtype=2), -2), (dict(Nq=129), -2), (dict(page=17), -2), (dict(scale=0.0), -1),
    (dict(scale=float("nan")), -1), (dict(width=1 << 28), -1), (dict(P=1 << 30), -1), (dict(o=P[7] + 8), -3),
    (dict(lens=P[6] + 1), -3), (dict(ws=None), -6), (dict(ws=WS + 128), -3), (dict(ws_bytes=100), -6),
    (dict(o=P[0]), -1), (dict(lse=P[7]), -1), (dict(ws=P[1]), -1)])
def test_decode_refuses(A, kw, code):
    base = dict(q=P[0], kc=P[1], vc=P[2], sk=P[3], sv=P[4], table=P[5], lens=P[6], o=P[7], lse=P[8], B=2, Nq=1, Hq=4,
                H=2, d=64, P=9, page=16, width=4, scale=0.125, causal=1, dtype=A.ATTN_BF16, ws=WS,
                ws_bytes=A.attn_kv8_decode_workspace_size(1, 4, 2, 64), stream=None)
    assert call(A.lib.attn_kv8_decode, DECODE, base, **kw) == code and A.last_error()


FWD = "q k v o lse cu_q cu_k B Tq Tk Hq Hkv d qs ks vs scale causal dtype ws ws_bytes stream"
BWD = ("q k v o lse dO dq dk dv cu_q cu_k B Tq Tk Hq Hkv d qs ks vs scale causal dtype ws ws_bytes stream")
SIZES = dict(B=3, Tq=100, Tk=120, Hq=4, Hkv=2, d=64, qs=256, ks=128, vs=128, scale=0.125, causal=1, dtype=0, stream=None)
COMMON = [
    (dict(q=None), -1), (dict(cu_q=None), -1), (dict(k=None), -1), (dict(B=0), -1), (dict(B=8193), -2),
    (dict(Tq=-1), -1), (dict(Tk=1 << 26), -1), (dict(Hq=5), -1), (dict(Hkv=0), -1), (dict(Hq=4096, Hkv=2, qs=1 << 18), -1),
    (dict(d=80), -2), (dict(dtype=5), -2), (dict(scale=-1.0), -1), (dict(scale=float("inf")), -1), (dict(qs=192), -1),
    (dict(ks=64), -1), (dict(vs=160), -1), (dict(qs=1 << 30), -1), (dict(cu_k=P[10] + 2), -3), (dict(v=P[2] + 8), -3)]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(o=P[0]), -1), (dict(lse=P[3]), -1), (dict(lse=P[9]), -1)])
def test_varlen_fwd_refuses(A, kw, code):
    base = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], cu_q=P[9], cu_k=P[10], ws=None, ws_bytes=0, **SIZES)
    assert call(A.lib.attn_varlen_fwd, FWD, base, **kw) == code and A.last_error()


@pytest.mark.parametrize("kw,code", [(dict(ws=None), -6), (dict(ws_bytes=1000), -6), (dict(ws=WS + 16), -3),
                                     (dict(ws=P[1]), -1), (dict(o=WS), -1)])
def test_varlen_fwd_refuses_its_workspace(A, kw, code):
    """Few queries on many keys: a workspace is needed."""
    sizes = {**SIZES, "Tk": 50000}
    need = A.attn_varlen_fwd_workspace_size(3, 100, 50000, 4, 2, 64)
    assert need > 0
    base = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], cu_q=P[9], cu_k=P[10], ws=WS, ws_bytes=need, **sizes)
    assert call(A.lib.attn_varlen_fwd, FWD, base, **kw) == code and A.last_error()


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dO=None), -1), (dict(dv=None), -1), (dict(dq=P[6] + 4), -3), (dict(ws=None), -6), (dict(ws_bytes=1000), -6),
    (dict(ws=WS + 16), -3), (dict(dq=P[5]), -1), (dict(dk=P[8]), -1), (dict(ws=P[3]), -1)])
def test_varlen_bwd_refuses(A, kw, code):
    base = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], dO=P[5], dq=P[6], dk=P[7], dv=P[8], cu_q=P[9], cu_k=P[10],
                ws=WS, ws_bytes=A.attn_varlen_bwd_workspace_size(3, 100, 4, 2, 64), **SIZES)
    assert call(A.lib.attn_varlen_bwd, BWD, base, **kw) == code and A.last_error()


def test_nothing_to_do_is_no_error(A):
    """No rows: nothing is enqueued (and no device is needed)."""
    base = dict(q=None, k=None, v=None, o=None, lse=None, cu_q=P[9], cu_k=P[10], ws=None, ws_bytes=0,
                **{**SIZES, "Tq": 0, "Tk": 0})
    assert call(A.lib.attn_varlen_fwd, FWD, base) == 0
    base.update(dO=None, dq=None, dk=None, dv=None)
    assert call(A.lib.attn_varlen_bwd, BWD, base) == 0
    assert A.lib.attn_kv8_append(None, None, 0, 0, None, 0, 1, 64, None, None, None, None, 1, 16, 0, None) == 0


def test_workspace_sizes(A):
    f = A.attn_varlen_bwd_workspace_size
    assert f(0, 10, 1, 1, 64) == 0 and f(1, -1, 1, 1, 64) == 0 and f(1, 10, 0, 1, 64) == 0
    assert f(1, 10, 1, 1, 96) == 0 and f(1, 10, 3, 2, 64) == 0
    # three fp32 parts over every head's rows, padded by at most 64 a sequence
    assert f(5, 1000, 8, 8, 128) >= 8 * 1000 * (128 + 2) * 4
    assert f(5, 1000, 8, 8, 128) <= 8 * (1000 + 5 * 64) * (128 + 2) * 4 + 4096
    # and, where key tiles may be split, a fixed number of partial dK, dV tiles
    assert f(1, 100000, 2, 1, 64) - 2 * 100000 * (64 + 2) * 4 <= 608 * 2 * 128 * 64 * 4 + 100000
    h = A.attn_varlen_fwd_workspace_size
    assert h(4, 8192, 8192, 16, 4, 128) == 0 and h(1, 64, 500, 12, 4, 64) == 0  # enough query tiles; few keys
    assert 0 < h(1, 64, 100000, 12, 4, 64) <= 2 * 152 * 2 * 128 * 66 * 4
    g = A.attn_kv8_decode_workspace_size
    assert g(0, 1, 1, 64) == 0 and g(1, 3, 2, 64) == 0 and g(1, 2, 2, 60) == 0 and g(1, 8, 1, 128) > 0


def test_conveniences_refuse_other_tensors(A):
    """CPU tensors, wrong types, shapes and strides raise before the library is called."""
    z = torch.zeros
    with pytest.raises(ValueError):
        A.varlen_fwd(z(4, 2, 64).half(), z(4, 2, 64).half(), z(4, 2, 64).half(), z(2).int(), z(2).int())
    with pytest.raises(ValueError):
        A.kv8_append(z(4, 2, 64).half(), z(4, 2, 64).half(), z(4).long(), z(3, 2, 16, 64).byte(),
                     z(3, 2, 16, 64).byte(), z(3, 2), z(3, 2))
    with pytest.raises(ValueError):
        A.kv8_decode(z(1, 1, 2, 64).half(), z(3, 2, 16, 64).byte(), z(3, 2, 16, 64).byte(), z(3, 2), z(3, 2),
                     z(1, 4).int(), z(1).int())
    with pytest.raises(ValueError):
        A.pages_extend(z(3).int(), z(3).int(), z(3, 4).int(), z(9).int(), z(1).int(), 16, 3)
    with pytest.raises(ValueError):
        A.pages_release(z(3).int(), z(3).int(), z(3, 4).int(), z(9).int(), z(1).int(), 16)


@pytest.mark.parametrize("width,page", [((1 << 27) - 1, 16), ((1 << 27) - 7, 16), ((1 << 26) - 3, 32), ((1 << 25) - 1, 64)])
def test_decode_refuses_lengths_that_do_not_round_up(A, width, page):
    """Tables of more than 2^31 - 128 tokens: the last tile's end would not fit 32 bits."""
    assert (1 << 31) - 128 < width * page < 1 << 31
    base = dict(q=P[0], kc=P[1], vc=P[2], sk=P[3], sv=P[4], table=P[5], lens=P[6], o=P[7], lse=P[8], B=1, Nq=1, Hq=4,
                H=2, d=64, P=9, page=page, width=width, scale=0.125, causal=1, dtype=A.ATTN_BF16, ws=WS,
                ws_bytes=A.attn_kv8_decode_workspace_size(1, 4, 2, 64), stream=None)
    assert call(A.lib.attn_kv8_decode, DECODE, base) == -1 and "width * page" in A.last_error()
