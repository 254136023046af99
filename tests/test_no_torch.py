"""Planning through the binding needs no torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PLAN = """
import sys
sys.modules["torch"] = None  # every import of it fails
from types import SimpleNamespace
from persistent_megakernel_decode_gb300 import build, runtime as rt
build.build()
shape = SimpleNamespace(L=2, H=256, Hq=4, Hkv=2, D=64, F=512, V=1024, qk_norm=False, eps=1e-5, theta=1e4)
p = rt.Plan.llama(shape, 1, [10], 2, 16, num_sms=152, smem_per_cta=232448)
q, ids, th, tasks = p.export()
assert p.info()["num_tasks"] == len(tasks) > 0
p.free()
"""


def test_plans_without_torch():
    r = subprocess.run([sys.executable, "-c", PLAN], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
