"""The binding's C part is loaded by the calls that need it, and belongs to one
Python ABI.  No GPU."""
import importlib.machinery
import os
import shutil
import subprocess
import sys

import pytest

from layers_proj_rms_gb300 import build as B

CODE = """
import torch, layers_proj_rms_gb300 as M
x = torch.zeros(2, 4, 4)
try:
    M.mhc_sinkhorn_fwd(x, x, 3, 1e-6)
except ValueError as e:
    print("older:", e)
assert M.mhc_moe_rows(10, 2, 4, 8) == 48
ids = torch.zeros(2, 2, dtype=torch.int32)
for _ in range(2):
    try:
        M.mhc_moe_sort(ids, 1, ids, ids, ids, ids)
    except ImportError as e:
        print("edge:", e)
"""


def test_the_other_operators_do_without_it(tmp_path):
    B.build()
    pkg = tmp_path / "layers_proj_rms_gb300"
    shutil.copytree(B.HERE, pkg, ignore=shutil.ignore_patterns("_build", "__pycache__", "csrc"))
    os.makedirs(pkg / "_build")
    os.symlink(B.LIB, pkg / "_build" / "libmhc.so")
    r = subprocess.run([sys.executable, "-c", CODE], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)}, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.splitlines()
    assert lines[0].startswith("older:") and "CUDA" in lines[0]
    # found missing at every such call, by name
    assert len(lines) == 3 and all(s.startswith("edge:") and "_marshal" in s for s in lines[1:])


def test_its_name_says_for_which_python():
    B.build()
    suffix = importlib.machinery.EXTENSION_SUFFIXES[0]
    assert "cpython" in suffix and os.path.basename(B.MARSHAL) == "_marshal" + suffix
    assert os.path.exists(B.MARSHAL)


def test_a_build_without_python_headers_says_so(tmp_path, monkeypatch):
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "m.so"))
    monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.warns(UserWarning, match="Python.h"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.MARSHAL)
