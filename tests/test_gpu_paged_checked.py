"""The paged cache's tests of far pages, long lines, outgrown workspaces, positions and waits that give up on the
checked build, whose kernels look at every index before they use it."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_on_the_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from cross_model_kv_gb300 import build
    build.build(checked=True)
    files = [f"tests/test_gpu_paged_{x}.py" for x in ("positions", "line", "workspace", "far", "ends")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files],
                       cwd=ROOT, env=dict(os.environ, KVB_LIBRARY="checked"), capture_output=True, text=True, timeout=600)
    if r.returncode != 0 or " passed" not in r.stdout:
        pytest.fail(r.stdout[-6000:] + r.stderr[-2000:])
