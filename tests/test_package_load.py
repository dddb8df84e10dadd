"""Loading the package without the Python extension of the bounded-cache operators, or beside one
that was built for another PyTorch; building it again by the command that the error names."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "paged_kv_cache_204_gb300"
CALL = """
import torch
import paged_kv_cache_204_gb300 as pkv
from paged_kv_cache_204_gb300.block_manager import BlockManager
bm = BlockManager(8, 16)
assert pkv.decode_workspace_bytes(4, 8, 64, 100) > 0
t = torch.zeros(1, 2, dtype=torch.int32)
try:
    pkv.paged_attention_decode_window(t, t, t, t, t, t, 1.0, 4, 0, 32, t)
except Exception as e:
    print(type(e).__name__, e)
"""


@pytest.fixture
def tree(tmp_path):
    """A copy of the package and what it is built from, with the times of the originals."""
    import __graft_entry__
    __graft_entry__.build()
    for d in (NAME, "include"):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d, ignore=shutil.ignore_patterns("*.o", "__pycache__"))
    return tmp_path


def call(tree):
    r = subprocess.run([sys.executable, "-c", CALL], cwd=tree, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tree)})
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


def test_as_built(tree):
    assert call(tree).startswith("ValueError")  # the extension's own check of its arguments


def test_missing_extension_fails_the_calls_that_need_it_only(tree):
    os.remove(tree / NAME / "_build" / "_pkv_torch.so")
    said = call(tree)
    assert said.startswith("ImportError") and "missing" in said
    command = re.search("`(.*)`", said).group(1).split()
    assert command[0] == "python" and os.path.samefile(command[1], tree / NAME / "build.py")
    before = os.stat(tree / NAME / "_build" / "libpkv.so").st_mtime_ns
    subprocess.run([sys.executable] + command[1:], cwd="/", check=True, capture_output=True)
    assert os.stat(tree / NAME / "_build" / "libpkv.so").st_mtime_ns == before  # that one was up to date
    assert call(tree).startswith("ValueError")


def test_extension_of_another_torch_is_not_loaded(tree):
    abi = tree / NAME / "_build" / "_pkv_torch.so.abi"
    abi.write_text("torch 1.0 cpython-30")
    said = call(tree)
    assert said.startswith("ImportError") and "was built for torch 1.0 cpython-30" in said and "build.py" in said
    check = "import build; print(build.library_up_to_date(), build.binding_up_to_date(), build.up_to_date())"
    r = subprocess.run([sys.executable, "-c", check], cwd=tree / NAME, capture_output=True, text=True)
    assert r.stdout.split() == ["True", "False", "False"], r.stderr
