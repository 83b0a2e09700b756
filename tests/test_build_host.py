"""What is built, when it is built again, and what the dense calls need of it (no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "exact_tiled_attention_22_gb300"


@pytest.fixture()
def copy(tmp_path):
    """The package with both libraries, to take parts away from."""
    from exact_tiled_attention_22_gb300 import build
    build.build()
    shutil.copytree(os.path.join(ROOT, PKG), tmp_path / PKG, ignore=shutil.ignore_patterns("__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    os.makedirs(tmp_path / "_build")
    shutil.copy(os.path.join(ROOT, "_build", "attn_bind.stamp"), tmp_path / "_build")
    return tmp_path


def python(where, code):
    return subprocess.run([sys.executable, "-c", code], cwd=where, capture_output=True, text=True, timeout=120)


@pytest.mark.parametrize("broken", [False, True])
def test_dense_calls_do_not_need_the_binding(copy, broken):
    """Without attn_bind.so, or with one that does not load, the package imports and the
    C ABI answers; the packed and serving calls raise."""
    so = copy / PKG / "attn_bind.so"
    so.write_text("no library") if broken else so.unlink()
    r = python(copy, f"""
from {PKG} import attn
assert attn.__file__.startswith({str(copy)!r})
assert attn.attn_bwd_workspace_size(1, 1, 128, 64) > 0
for _ in range(2):
    try:
        attn.pages_release(None, None, None, None, None, 16)
    except (RuntimeError, ImportError) as e:
        assert "attn_bind.so" in str(e), e
    else:
        raise SystemExit("no error")
""")
    assert r.returncode == 0, r.stderr


def test_the_binding_is_built_again_for_another_torch(copy):
    """Another torch, Python or toolkit than the module was built for: attn_bind.so is
    built again, libattn.so, which does not know them, is not."""
    r = python(copy, f"""
import os
from {PKG} import build
assert build.up_to_date()
old = os.stat(build.LIB).st_mtime_ns
with open(build.STAMP) as f:
    kept = f.read()
assert kept == build._stamp() and "version" in kept
for text in (kept.replace("version", "another version", 1), None):
    if text is None:
        os.remove(build.STAMP)
    else:
        with open(build.STAMP, "w") as f:
            f.write(text)
    assert build.lib_up_to_date() and not build.bind_up_to_date() and not build.up_to_date()
did = []
build.compile_bind = lambda obj: did.append("compile")
build.link_bind = lambda obj: did.append("link")
build.build()
assert did == ["compile", "link"] and os.stat(build.LIB).st_mtime_ns == old
""")
    assert r.returncode == 0, r.stderr


def test_libattn_is_in_place_before_the_binding_fails(copy):
    """A torch without C++ headers: build() says so, and the dense calls have their library."""
    r = python(copy, f"""
import os
from {PKG} import build
os.remove(build.LIB)
os.remove(build.BIND)
build.SOURCES[:] = ["attn_diag.cu"]  # (one small file stands for them all)
def fail(obj):
    raise RuntimeError("no headers")
build.compile_bind = fail
try:
    build.build()
except RuntimeError as e:
    assert "no headers" in str(e)
else:
    raise SystemExit("no error")
assert os.path.exists(build.LIB) and not os.path.exists(build.BIND) and build.lib_up_to_date()
""")
    assert r.returncode == 0, r.stderr
