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
