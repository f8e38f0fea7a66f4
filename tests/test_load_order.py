"""The library and torch in one process, whichever is asked for first (CPU only)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import weight_quantization_amd as wq
assert wq.hlwq_packed_bytes(1, 128, bits=5) == 80  # loads the library
import torch
print(*sorted({l.split()[-1] for l in open("/proc/self/maps") if "libamdhip64" in l}))
"""


def test_one_hip_runtime_where_the_library_is_used_before_torch():
    pytest.importorskip("torch")
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert len(r.stdout.split()) == 1, r.stdout
