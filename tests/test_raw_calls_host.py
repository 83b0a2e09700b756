"""The packed and serving entry points of attn.py that mirror the C ABI: same names, same
order and types of arguments as include/attn.h, passed on as they are given (no GPU)."""
import ctypes
import inspect
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"int": ctypes.c_int, "long long": ctypes.c_longlong, "size_t": ctypes.c_size_t, "float": ctypes.c_float,
         "attn_dtype_t": ctypes.c_int}


def prototypes():
    with open(os.path.join(ROOT, "include", "attn.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    for ret, name, args in re.findall(r"(int|size_t) (attn_(?:pages|kv8|varlen)\w+)\((.*?)\);", text, re.S):
        split = [re.match(r"\s*(.*?)(\w+)\s*$", a, re.S).groups() for a in args.split(",")]
        yield name, ret, [(n, ctypes.c_void_p if "*" in t else TYPES[t.replace("const", "").strip()]) for t, n in split]


PROTOTYPES = list(prototypes())


@pytest.fixture(scope="module")
def A():
    from exact_tiled_attention_22_gb300 import build
    build.build()
    from exact_tiled_attention_22_gb300 import attn
    return attn


def test_all_are_there():
    assert len(PROTOTYPES) == 9


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
