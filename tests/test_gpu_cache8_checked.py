"""The 8-bit cache's edge, workspace and long-line tests on the checked build, whose
kernels look at every index before they use it: tokens, rows, blocks and slots of the
cache, entries of the page table, units and slots of the workspace."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_edges_and_long_lines_on_the_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from cross_model_kv_gb300 import build
    build.build(checked=True)
    files = [f"tests/test_gpu_cache8_{n}.py" for n in ("bounds", "workspace", "long")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files],
                       cwd=ROOT, env=dict(os.environ, KVB_LIBRARY="checked"), capture_output=True, text=True, timeout=900)
    if r.returncode != 0 or " passed" not in r.stdout:
        pytest.fail(r.stdout[-6000:] + r.stderr[-2000:])
