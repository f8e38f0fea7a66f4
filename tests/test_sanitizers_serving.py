"""Host code of the serving operators under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): built with both,
failing on the first report (device code is compiled as usual and never launched), and driven by the plain C client
tests/serving_abi_check.c, which also shows that include/hlwq_attention.h is C99."""
import os
import subprocess

import pytest

from test_sanitizers import CLANG, ROOT, _env
from weight_quantization_amd import build as wqb


def test_serving_validation_under_sanitizers(tmp_path):
    if not os.path.exists(CLANG):
        pytest.skip("no ROCm clang")
    if not os.path.exists(os.path.join(wqb.BUILD, "hlwq_tables.inc")):
        wqb.generate_tables()
    lib = str(tmp_path / "libserving_asan.so")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-g"]
    r = subprocess.run([wqb._hipcc(), *wqb.HIPCC_FLAGS, *san, "-I", wqb.INCLUDE, "-I", wqb.BUILD,
                        *(os.path.join(wqb.CSRC, s) for s in wqb.SERVING_SOURCES), "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    exe = str(tmp_path / "serving_abi_asan")
    subprocess.run([CLANG, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", wqb.INCLUDE, os.path.join(ROOT, "tests", "serving_abi_check.c"),
                    "-L", str(tmp_path), "-lserving_asan", "-Wl,-rpath," + str(tmp_path), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=_env())
    assert r.returncode == 0, r.stderr[-4000:]
    assert "serving abi ok" in r.stdout
