"""The compiled binding of the paged-cache calls: its file belongs to one torch and one Python, and the calls that do
not need it work where it is missing."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def build():
    from block_sparse_long_09_b200 import build as b
    b.build()
    return b


def test_file_is_of_this_torch_and_python(build, monkeypatch):
    import sysconfig
    path = build.binding_path()
    assert torch.__version__ in path and sysconfig.get_config_var("SOABI") in path
    assert os.path.exists(path) and not build.needs_build(path)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert build.binding_path() != path and build.needs_build(build.binding_path())


def test_calls_without_the_binding(build, tmp_path):
    """A copy of the package with the library alone: the import and the ctypes calls work, a paged-cache call says
    what is missing."""
    pkg = tmp_path / "block_sparse_long_09_b200"
    pkg.mkdir()
    src = os.path.join(ROOT, "block_sparse_long_09_b200")
    for f in os.listdir(src):
        if f.endswith(".py") or f == "libqsa.so":
            os.symlink(os.path.join(src, f), pkg / f)
    child = textwrap.dedent("""
        import torch
        from block_sparse_long_09_b200 import qsa
        assert qsa.LIB_PATH.startswith({root!r}), qsa.LIB_PATH
        assert qsa.workspace_size(qsa.OP_CHUNK_PAGED, 1, 1) > 0 and qsa.default_config().head_dim == 256
        x = torch.zeros(1)
        for call in (lambda: qsa.rope_axes(x, x, x, (1, 1, 1)),
                     lambda: qsa.cache_write_paged(x, x, x, x, x, x, x),
                     lambda: qsa.cache_read_paged(x, x, x, x, x, 1),
                     lambda: qsa.chunk_attn_paged(x, x, x, x, x, x, 1)):
            try:
                call()
                raise SystemExit("no error")
            except ImportError as e:
                assert "block_sparse_long_09_b200.build" in str(e), e
        print("CHILD-OK")
    """).format(root=str(tmp_path))
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    p = subprocess.run([sys.executable, "-c", child], cwd=tmp_path, env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "CHILD-OK" in p.stdout, p.stdout + p.stderr[-3000:]
