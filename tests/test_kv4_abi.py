"""What the calls on the 4-bit cache and the read of a cache refuse on the host, before any device
work, and that attn.py passes their arguments on in the C ABI's order (no GPU needed)."""
import ctypes
import inspect
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def A():
    from exact_tiled_attention_22_gb300 import build
    build.build()
    from exact_tiled_attention_22_gb300 import attn
    return attn


# Fake aligned addresses, far apart: every call below is refused on the host.
P = [0x100000000 * (i + 1) for i in range(20)]
WS = 1 << 44
TYPES = {"int": ctypes.c_int, "long long": ctypes.c_longlong, "size_t": ctypes.c_size_t, "float": ctypes.c_float,
         "attn_dtype_t": ctypes.c_int}


def prototypes():
    with open(os.path.join(ROOT, "include", "attn.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    for ret, name, args in re.findall(r"(int|size_t) (attn_kv(?:4|_)\w+)\((.*?)\);", text, re.S):
        split = [re.match(r"\s*(.*?)(\w+)\s*$", a, re.S).groups() for a in args.split(",")]
        yield name, ret, [(n, ctypes.c_void_p if "*" in t else TYPES[t.replace("const", "").strip()]) for t, n in split]


PROTOTYPES = list(prototypes())


@pytest.mark.parametrize("name,ret,args", PROTOTYPES, ids=[p[0] for p in PROTOTYPES])
def test_arguments_reach_the_library_in_order(A, monkeypatch, name, ret, args):
    fn = getattr(A.lib, name)
    assert list(fn.argtypes) == [t for _, t in args] and fn.restype == TYPES[ret]
    wrapper = getattr(A, name)
    assert list(inspect.signature(wrapper).parameters) == [n for n, _ in args]
    given = [A.ATTN_BF16 if n == "dtype" else (i % 2 if n == "causal" else (0.5 if n == "scale" else 1000 + i))
             for i, (n, _) in enumerate(args)]
    got = []

    class Lib:
        def __getattr__(self, called):
            assert called == name
            return lambda *a: got.append(list(a)) or 0

    monkeypatch.setattr(A, "lib", Lib())
    assert wrapper(*given) == 0
    assert got == [given]


def call(fn, names, base, kw):
    args = dict(base)
    assert not set(kw) - set(args)
    args.update(kw)
    return fn(*(args[n] for n in names.split()))


CACHE = [(dict(kc=None), -1), (dict(sv=None), -1), (dict(H=0), -1), (dict(P=0), -1), (dict(d=96), -2), (dict(dtype=3), -2),
         (dict(page=24), -2), (dict(page=256), -2), (dict(P=1 << 30, H=2), -1), (dict(kc=P[3] + 16), -3),
         (dict(vc=P[4] + 8), -3), (dict(sk=P[5] + 8), -3), (dict(sv=P[6] + 2), -3)]

APPEND = "k v ks vs slots T H d kc vc sk sv P page dtype stream"


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(k=None), -1), (dict(slots=None), -1), (dict(T=-1), -1), (dict(T=1 << 29), -1), (dict(T=1 << 31), -1),
    (dict(ks=120), -1), (dict(vs=132), -1), (dict(ks=1 << 32), -1), (dict(v=P[1] + 8), -3), (dict(slots=P[2] + 4), -3),
    (dict(kc=P[0]), -1), (dict(vc=P[3]), -1), (dict(sk=P[2]), -1), (dict(sv=P[5] + 16), -1), (dict(sk=P[3] + 9000), -3),
    (dict(sk=P[3] + 9 * 2 * 16 * 32 - 16), -1)])
def test_append_refuses(A, kw, code):
    base = dict(k=P[0], v=P[1], ks=128, vs=128, slots=P[2], T=5, H=2, d=64, kc=P[3], vc=P[4], sk=P[5], sv=P[6], P=9,
                page=16, dtype=A.ATTN_F16, stream=None)
    assert call(A.lib.attn_kv4_append, APPEND, base, kw) == code and A.last_error()


READ = "kc vc sk sv table lens cu k v B T H d P page width bits dtype stream"


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(table=None), -1), (dict(lens=None), -1), (dict(cu=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(B=0), -1), (dict(width=0), -1), (dict(T=-1), -1), (dict(T=1 << 31), -1), (dict(width=1 << 27), -1),
    (dict(bits=5), -2), (dict(k=P[7] + 8), -3), (dict(cu=P[9] + 2), -3), (dict(table=P[1] + 1), -3),
    (dict(k=P[8]), -1), (dict(k=P[3]), -1), (dict(v=P[9]), -1), (dict(v=P[1]), -1)])
def test_read_refuses(A, kw, code):
    base = dict(kc=P[3], vc=P[4], sk=P[5], sv=P[6], table=P[1], lens=P[2], cu=P[9], k=P[7], v=P[8], B=3, T=40, H=2, d=64,
                P=9, page=16, width=4, bits=4, dtype=A.ATTN_F16, stream=None)
    assert call(A.lib.attn_kv_read, READ, base, kw) == code and A.last_error()


def test_read_of_the_8_bit_cache_refuses(A):
    base = dict(kc=P[3] + 16, vc=P[4], sk=P[5] + 4, sv=P[6], table=P[1], lens=P[2], cu=P[9], k=P[7], v=P[8], B=3, T=40, H=2,
                d=64, P=9, page=16, width=4, bits=8, dtype=A.ATTN_F16, stream=None)
    for kw, code in ((dict(kc=P[3] + 8), -3), (dict(sk=P[5] + 2), -3), (dict(k=P[3]), -1)):
        assert call(A.lib.attn_kv_read, READ, base, kw) == code and A.last_error()


def test_nothing_to_do_is_no_error(A):
    """No rows: nothing is enqueued (and no device is needed)."""
    assert A.lib.attn_kv4_append(None, None, 0, 0, None, 0, 1, 64, None, None, None, None, 1, 16, 0, None) == 0
    for bits in (4, 8):
        assert A.lib.attn_kv_read(P[3], P[4], P[5], P[6], P[1], P[2], P[9], None, None, 3, 0, 2, 64, 9, 16, 4, bits, 0,
                                  None) == 0


def test_conveniences_refuse_other_tensors(A):
    """CPU tensors and types that are no 16-bit floats raise before the library is called."""
    z = torch.zeros
    kc, ks = z(3, 2, 16, 32).byte(), z(3, 2, 16, 2).bfloat16()
    with pytest.raises(ValueError):
        A.kv4_append(z(4, 2, 64).half(), z(4, 2, 64).half(), z(4).long(), kc, kc, ks, ks)
    for dtype in (torch.float16, torch.float32):
        with pytest.raises(ValueError):
            A.kv4_read(kc, kc, ks, ks, z(1, 4).int(), z(1).int(), z(2).int(), 3, dtype)
        with pytest.raises(ValueError):
            A.kv8_read(z(3, 2, 16, 64).byte(), z(3, 2, 16, 64).byte(), z(3, 2), z(3, 2), z(1, 4).int(), z(1).int(),
                       z(2).int(), 3, dtype)


DECODE = "q kc vc sk sv table lens o lse B Nq Hq H d P page width scale causal dtype ws ws_bytes stream"


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(q=None), -1), (dict(table=None), -1), (dict(lse=None), -1), (dict(B=0), -1), (dict(Nq=0), -1), (dict(Hq=3), -1),
    (dict(Hq=0), -1), (dict(Nq=129), -2), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(width=1 << 27), -1), (dict(width=(1 << 27) - 15), -1), (dict(width=0), -1),
    (dict(B=1 << 29), -1), (dict(Hq=1 << 25), -1), (dict(o=P[7] + 8), -3), (dict(lens=P[2] + 1), -3), (dict(ws=None), -6),
    (dict(ws=WS + 128), -3), (dict(ws_bytes=100), -6), (dict(o=P[0]), -1), (dict(lse=P[7]), -1), (dict(ws=P[3]), -1),
    (dict(o=P[5]), -1)])
def test_decode_refuses(A, kw, code):
    base = dict(q=P[0], kc=P[3], vc=P[4], sk=P[5], sv=P[6], table=P[1], lens=P[2], o=P[7], lse=P[8], B=2, Nq=1, Hq=4,
                H=2, d=64, P=9, page=16, width=4, scale=0.125, causal=1, dtype=A.ATTN_BF16, ws=WS,
                ws_bytes=A.attn_kv4_decode_workspace_size(1, 4, 2, 64), stream=None)
    assert call(A.lib.attn_kv4_decode, DECODE, base, kw) == code and A.last_error()


def test_decode_workspace_sizes(A):
    f = A.attn_kv4_decode_workspace_size
    assert f(0, 1, 1, 64) == 0 and f(1, 3, 2, 64) == 0 and f(1, 2, 2, 60) == 0 and f(129, 1, 1, 64) == 0
    assert 0 < f(1, 4, 1, 64) < f(1, 8, 1, 64) < f(1, 16, 1, 64) == f(128, 64, 1, 64) < f(1, 16, 1, 128)


def test_decode_convenience_refuses_other_tensors(A):
    z = torch.zeros
    kc, ks = z(3, 2, 16, 32).byte(), z(3, 2, 16, 2).bfloat16()
    with pytest.raises(ValueError):
        A.kv4_decode(z(1, 1, 2, 64).half(), kc, kc, ks, ks, z(1, 4).int(), z(1).int())
