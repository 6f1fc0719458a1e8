"""The C hand-off module on a torch without DLPack's exchange functions: the matmul's call as ever, the cache's refused."""
import importlib.machinery
import importlib.util
import shutil
import subprocess

import pytest

import bit_quantized_gemm_qmm_b200 as q
from bit_quantized_gemm_qmm_b200 import _build, kv


@pytest.mark.parametrize("header", [None, "#define DLPACK_MAJOR_VERSION 1\n#define DLPACK_MINOR_VERSION 0\n", "typedef int DLTensor;\n"])
def test_builds_without_exchange_functions(tmp_path, monkeypatch, header):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    includes = []
    if header is not None:
        (tmp_path / "include" / "ATen").mkdir(parents=True)
        (tmp_path / "include" / "ATen" / "dlpack.h").write_text(header)
        includes = [str(tmp_path / "include")]
    out = str(tmp_path / "_qmm_call.so")
    subprocess.run(_build.call_command(cc, out, includes), check=True)
    loader = importlib.machinery.ExtensionFileLoader("_qmm_call", out)
    m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_qmm_call", out, loader=loader))
    loader.exec_module(m)
    assert callable(m.bind) and callable(m.qmm_ex) and not hasattr(m, "bind_kv")
    with pytest.raises(TypeError):
        m.qmm_ex(1)
    monkeypatch.setattr(kv, "_call", None)
    monkeypatch.setattr(q, "_qmm_call", m, raising=False)
    monkeypatch.setattr(q, "lib", lambda: object())
    with pytest.raises(q.QmmUnavailable, match="exchange functions"):
        kv._calls()
