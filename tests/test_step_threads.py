"""The step planner's host code entered by two threads at once.  CPU only: the
runtime's calls are stood in for."""

import os
import subprocess

from paged_kv_cache_124_gb300 import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_plans_of_different_sizes_from_two_threads():
    """tests/step_threads_check.cu: no call lowers the shared-memory limit that another's launch relies on."""
    out_dir = os.path.join(ROOT, "_build", "step_threads")
    os.makedirs(out_dir, exist_ok=True)
    exe = os.path.join(out_dir, "step_threads_check")
    r = subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-cudart", "shared", "-I", b.INCLUDE, "-I", b.CSRC,
                        os.path.join(ROOT, "tests", "step_threads_check.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    cuda = os.path.join(os.path.dirname(os.path.dirname(b._nvcc())), "lib64")
    env = dict(os.environ, LD_LIBRARY_PATH=os.pathsep.join([cuda, os.environ.get("LD_LIBRARY_PATH", "")]))
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
