"""Host code of the operators for drafted tokens and experts under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only),
driven by the plain C client tests/drafts_abi_check.c, which also shows that their headers are C99; and the loads to LDS that
the experts' kernels write in assembly."""
import os
import re
import subprocess

import pytest

from test_sanitizers import CLANG, ROOT, _env
from weight_quantization_amd import build as wqb


@pytest.fixture(autouse=True)
def tables():
    if not os.path.exists(os.path.join(wqb.BUILD, "hlwq_tables.inc")):
        wqb.generate_tables()


def test_validation_under_sanitizers(tmp_path):
    if not os.path.exists(CLANG):
        pytest.skip("no ROCm clang")
    lib = str(tmp_path / "libserving_asan.so")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-g"]
    r = subprocess.run([wqb._hipcc(), *wqb.HIPCC_FLAGS, *san, "-I", wqb.INCLUDE, "-I", wqb.BUILD,
                        *(os.path.join(wqb.CSRC, s) for s in wqb.SERVING_SOURCES), "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    exe = str(tmp_path / "drafts_abi_asan")
    subprocess.run([CLANG, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", wqb.INCLUDE, os.path.join(ROOT, "tests", "drafts_abi_check.c"),
                    "-L", str(tmp_path), "-lserving_asan", "-Wl,-rpath," + str(tmp_path), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=_env())
    assert r.returncode == 0, r.stderr[-4000:]
    assert "drafts abi ok" in r.stdout


def test_loads_to_lds_bring_their_wait_states(tmp_path):
    out = str(tmp_path / "moe.s")
    flags = [f for f in wqb.HIPCC_FLAGS if f != "-shared"]
    subprocess.run([wqb._hipcc(), *flags, "--cuda-device-only", "-S", "-I", wqb.INCLUDE, "-I", wqb.BUILD,
                    os.path.join(wqb.CSRC, "moe.hip"), "-o", out], check=True, capture_output=True)
    found = 0
    for block in re.findall(r"#ASMSTART(.*?);;#ASMEND", open(out).read(), re.S):
        lines = [x.strip() for x in block.split("\n") if x.strip()]
        loads = [x for x in lines if re.search(r"_load_lds_|_load_\S+ .*\blds$", x)]
        if not loads:
            continue
        found += 1
        # M0, then the load alone; one wait state for M0, five for a scalar register that a VALU instruction wrote right before
        assert lines[-1] == loads[0] and lines[0].startswith("s_mov_b32 m0,"), lines
        waits = sum(int(x.split()[1]) + 1 if x.startswith("s_nop") else 1 for x in lines[1:-1])
        assert waits >= 1 and (waits + 1 >= 5 or not re.search(r"\bs(\[|\d)", loads[0])), lines
    assert found >= 32  # both bits, both banks
