"""A call's workspace is checked against the plan that it is launched with (no GPU needed)."""
import glob
import os
import subprocess

from medusa_speculative_decoding_02_gb300 import build as mbuild

SRC = os.path.join(mbuild.ROOT, "tests", "c", "paged_plan_once.cu")


def test_one_plan_a_call(tmp_path):
    mbuild.build()
    objects = sorted(glob.glob(os.path.join(mbuild.BUILD, "*.cu.o")))
    if len(objects) != len(mbuild.sources()):
        mbuild.build(force=True)
        objects = sorted(glob.glob(os.path.join(mbuild.BUILD, "*.cu.o")))
    rest = [o for o in objects if os.path.basename(o) != "paged_attention_tc.cu.o"]
    exe = str(tmp_path / "paged_plan_once")
    subprocess.run([mbuild.nvcc(), *mbuild.ARCH, *mbuild.FLAGS, "-cudart", "static", SRC, *rest, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
