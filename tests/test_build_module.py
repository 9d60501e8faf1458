"""The module of the serving calls is compiled for one torch: the build notices another one, the
binding does not use a module of another one, and without it only the serving calls fail."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from post_weight_quantization_gb300 import build as b

PACKAGE = os.path.dirname(os.path.abspath(b.__file__))

CHECK = """
import torch
%s
from post_weight_quantization_gb300 import gptq as g
assert g.gptq_version() > 0 and g.gptq_workspace_size(g.GPTQ_WS_FACTOR, 0, 256) > 0
cache = g.KVCache(torch.zeros((1, 1, 16 * 72), dtype=torch.uint8), 16, 1, 64)
K = torch.zeros((1, 1, 64))
try:
    g.gptq_kv_append(cache, K, K, torch.zeros(1, dtype=torch.int64))
except ImportError as e:
    print("refused:", e)
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    b.build()


def _run(root, before=""):
    return subprocess.run([sys.executable, "-c", CHECK % before], cwd=root, capture_output=True, text=True)


def test_without_the_module_the_rest_works(tmp_path):
    pkg = tmp_path / os.path.basename(PACKAGE)
    pkg.mkdir()
    for name in os.listdir(PACKAGE):
        if name.endswith(".py") or name == "libgptq.so":
            shutil.copy(os.path.join(PACKAGE, name), pkg)
    got = _run(tmp_path)
    assert got.returncode == 0, got.stderr
    assert got.stdout.startswith("refused:") and "--force" in got.stdout


def test_a_module_of_another_torch_is_not_used():
    got = _run(os.path.dirname(PACKAGE), "torch.__version__ = '0.1'")
    assert got.returncode == 0, got.stderr
    assert got.stdout.startswith("refused:") and "torch 0.1" not in got.stdout and "this is 0.1" in got.stdout


def test_build_notices_another_torch_or_compiler(monkeypatch):
    was = b._fingerprint()
    assert b._fingerprint() == was
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", torch.__version__ + ".1")
        assert b._fingerprint() != was
    with monkeypatch.context() as m:
        m.setenv("CXX", "another-compiler")
        assert b._fingerprint() != was
