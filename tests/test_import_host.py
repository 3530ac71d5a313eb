"""The package without torch: importing it, building the library and loading it need none."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["torch"] = None  # every import of it raises
import combine_device_resident_gb300 as A
from combine_device_resident_gb300 import build
build.build()
L = A.load_library()
cfg = A.make_config(8, 16, 64, 256, 2)
assert L.a2av_config_check(cfg) == 0 and L.a2av_recv_arena_rows(cfg) == 8 * 64 * 2
print("loaded")
"""


def test_the_package_needs_no_torch_to_be_imported():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.split() == ["loaded"], r.stderr[-2000:]
