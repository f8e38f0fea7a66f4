"""The loads from memory straight to LDS that are written in assembly bring the waits of their own that the compiler, which
does not see them, cannot add (CPU only: the assembly of the attention kernels is read, nothing is run)."""
import os
import re
import subprocess

from weight_quantization_amd import build as wqb


def test_loads_to_lds_bring_their_wait_states(tmp_path):
    if not os.path.exists(os.path.join(wqb.BUILD, "hlwq_tables.inc")):
        wqb.generate_tables()
    out = str(tmp_path / "attention.s")
    flags = [f for f in wqb.HIPCC_FLAGS if f != "-shared"]
    subprocess.run([wqb._hipcc(), *flags, "--cuda-device-only", "-S", "-I", wqb.INCLUDE, "-I", wqb.BUILD,
                    os.path.join(wqb.CSRC, "attention.hip"), "-o", out], check=True, capture_output=True)
    found = 0
    for block in re.findall(r"#ASMSTART(.*?);;#ASMEND", open(out).read(), re.S):
        lines = [x.strip() for x in block.split("\n") if x.strip()]
        loads = [x for x in lines if re.search(r"_load_lds_|_load_\S+ .*\blds$", x)]
        if not loads:
            continue
        found += 1
        assert lines[-1] == loads[0] and lines[0].startswith("s_mov_b32 m0,"), lines
        # wait states between M0's write and the load; one instruction is one, s_nop n is n + 1
        waits = sum(int(x.split()[1]) + 1 if x.startswith("s_nop") else 1 for x in lines[1:-1])
        assert waits >= 1, lines
        # a VALU write of a scalar register may stand right before the block: five to the load that reads it
        assert waits + 1 >= 5 or not re.search(r"\bs(\[|\d)", loads[0]), lines
    assert found > 100
