"""The extension module behind the paged and norm calls: what needs it, when it is built
again, and what it says when it cannot be loaded (no GPU needed)."""
import subprocess
import sys

import pytest

from structured_sparse_attention_fibonacci_b200 import build as sa_build

PKG = "structured_sparse_attention_fibonacci_b200"


@pytest.fixture(scope="module", autouse=True)
def _built():
    sa_build.build()


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=sa_build.ROOT, capture_output=True,
                          text=True, timeout=300)


def test_calls_through_ctypes_do_without_the_extension_module():
    """fwd(), bwd() and decode() load the library alone; a paged call says why the module fails."""
    r = _python(f"""
import sys
sys.modules["{PKG}._binding"] = None        # as one that cannot be imported
import torch
import {PKG} as sa
assert sa.lib().sparse_attn_workspace_size and sa.status_string(0)
assert sa.workspace_size((1, 1, 1, 64, 64), torch.bfloat16, backward=True, window=4) > 0
assert sa.qk_norm_workspace_size((1, 1, 2, 8, 64), (1, 1, 1, 8, 64)) > 0
for _ in range(2):
    try:
        sa.qk_norm_rope(None, None, None, None)
    except RuntimeError as e:
        assert "build" in str(e) and str(e.__cause__) in str(e), e
    else:
        raise AssertionError("no error")
""")
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("change", ["torch", "missing", "module", "nothing"])
def test_the_extension_module_is_built_again_for_another_torch(change, tmp_path, monkeypatch):
    """Stale for another torch or Python than it was built for, whatever its file's time; only
    then is it built."""
    for name in ("BINDING", "BINDING_FOR"):
        path = tmp_path / name
        path.write_text(sa_build._built_for())
        monkeypatch.setattr(sa_build, name, str(path))
    if change == "torch":
        (tmp_path / "BINDING_FOR").write_text("torch 0.0\n")
    elif change != "nothing":
        (tmp_path / {"missing": "BINDING_FOR", "module": "BINDING"}[change]).unlink()
    assert sa_build._stale(sa_build.BINDING) == (change != "nothing")
    built = []
    monkeypatch.setattr(sa_build, "_build_binding", lambda *a: built.append(1))
    sa_build.build()
    assert len(built) == (change != "nothing")
