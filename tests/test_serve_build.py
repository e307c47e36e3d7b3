"""What the serving calls' native module asks of everyone else: nothing (no GPU)."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "learnable_channel_permutation_amd")


def python(code, cwd):
    p = subprocess.run([sys.executable, "-c", code], cwd=cwd, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr
    return p.stdout


def test_the_package_works_without_the_serving_module(tmp_path):
    """Learning and deploying need liblcp.so alone; a serving call says what is missing."""
    shutil.copytree(PKG, tmp_path / "learnable_channel_permutation_amd",
                    ignore=shutil.ignore_patterns("_serve.so", "__pycache__", "csrc"))
    out = python('''
import torch
import learnable_channel_permutation_amd as lcp
assert lcp.lcp_xt_pitch(100) >= 100 and lcp.lcp_sparse_pack_bytes(64, 64)[0] > 0 and lcp.LayerSession
x, i = torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int32)
for call in (lambda: lcp.lcp_rope(x, x, x, i), lambda: lcp.PagedKVCache.empty(1, 16, 1, 64, device="cpu"),
             lambda: lcp.lcp_kv_append(None, x, x, i)):
    try:
        call()
    except ImportError as e:
        assert "_serve.so" in str(e) and "build.py" in str(e)
        print("told")
''', tmp_path)
    assert out.split() == ["told"] * 3


def test_the_package_imports_where_torch_has_no_raw_stream():
    """Those two names of torch are not public: without them the public ones serve."""
    out = python('''
import torch
del torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
import learnable_channel_permutation_amd as lcp
class S:
    cuda_stream = 77
torch.cuda.current_device = None
torch.cuda.current_stream = lambda device=None: S
lcp._lib._current_device = lambda: 0
print(lcp._lib._stream(), lcp._lib._stream(S))
''', ROOT)
    assert out.split() == ["77", "77"]


def test_the_library_is_built_where_the_serving_module_cannot_be(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    monkeypatch.setattr(b, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "liblcp.so"))
    monkeypatch.setattr(b, "BIND", str(tmp_path / "_serve.so"))
    (tmp_path / "_serve.so").write_text("an older build")
    flags = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    class Failed(Done):
        returncode, stderr = 1, "no such header"

    def run(cmd, **kw):
        if cmd[0] == "g++":
            flags.extend(cmd)
            return Failed
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return Done

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="bind.cpp"):
        b.build()
    assert (tmp_path / "liblcp.so").read_text() == "built"
    assert not (tmp_path / "_serve.so").exists()         # not one of another version
    import torch
    assert "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi() in flags
