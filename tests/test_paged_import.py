"""The paged memory's extension module is built against one PyTorch; without it
the package's other calls work, and the paged ones say what is missing."""

import os
import subprocess
import sys

import pytest

import test_library_cpu as base

CODE = """
import torch
import transformer_xl_relative_txl_gb300 as txl
assert txl.txl_version() >= 160 and txl.txl_status_string(0) == "TXL_OK"
assert txl.txl_relattn_paged_workspace_bytes(1, 1, 1, 64, torch.bfloat16) > 0
try:
    txl.txl_relattn_forward(*[torch.zeros(1, 1, 1, 64)] * 3, *[torch.zeros(1, 64)] * 4)
except ValueError:
    pass
z = torch.zeros(1, dtype=torch.int32)
for _ in range(2):
    try:
        txl.txl_pages_free(dict(table=z[None], start=z, rows=z, refs=z), 16, z)
    except ImportError as e:
        assert "_paged.so" in str(e) and "build.py" in str(e), e
    else:
        raise SystemExit("no ImportError")
"""


@pytest.mark.parametrize("binding", [None, b"", b"\x7fELF of another PyTorch"])
def test_without_the_module(tmp_path, binding):
    base._build_if_missing()
    pkg = tmp_path / "transformer_xl_relative_txl_gb300"
    pkg.mkdir()
    for name in ("__init__.py", "libtxl_relattn.so"):
        os.symlink(os.path.join(base.PKG, name), pkg / name)
    if binding is not None:
        (pkg / "_paged.so").write_bytes(binding)
    # (__init__.py finds the library beside itself, by the path it is imported from.)
    res = subprocess.run([sys.executable, "-c", CODE], cwd=tmp_path, capture_output=True, text=True,
                         env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert res.returncode == 0, res.stderr


def test_the_library_is_linked_first(monkeypatch, tmp_path):
    """A module that does not compile leaves the library built."""
    import importlib.util

    spec = importlib.util.spec_from_file_location("txl_build_order", os.path.join(base.PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    linked = []

    def refuse():
        raise RuntimeError("no Python headers")

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "_compile", lambda s, extra: (s, ""))
    monkeypatch.setattr(build, "_compile_binding", refuse)
    monkeypatch.setattr(build, "_link", lambda cmd, target: linked.append(target))
    with pytest.raises(RuntimeError, match="no Python headers"):
        build.build()
    assert linked == [build.LIB]
