"""What the decayed attention's inline assembly takes for granted about the code
around it, checked on the listing of the built kernels."""
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")


def test_m0_serves_the_loads_into_lds_alone(tmp_path):
    """The register cannot be named as changed by the assembly (the compiler
    reserves it), so nothing else may use it."""
    built = os.path.join(ROOT, "_build", "kda_decay.hip.o")
    if not (os.path.exists(built) and os.path.exists(OBJDUMP)):
        pytest.skip("no object file or no disassembler here")
    shutil.copy(built, tmp_path / "decay.o")
    subprocess.run([OBJDUMP, "--offloading", "decay.o"], cwd=tmp_path, check=True, stdout=subprocess.DEVNULL)
    code, = glob.glob(str(tmp_path / "decay.o.*gfx950"))
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", code], check=True, capture_output=True,
                          text=True).stdout
    lines = [ln.split("//")[0].strip() for ln in text.splitlines()]
    uses = [i for i, ln in enumerate(lines) if re.search(r"\bm0\b", ln)]
    loads = [i for i, ln in enumerate(lines) if re.match(r"buffer_load\S* .*\blds\b", ln)]
    assert uses and len(uses) == len(loads)
    for i in uses:
        assert re.match(r"s_mov_b32 m0, ", lines[i]) and lines[i + 1] == "s_nop 0" and i + 2 in loads, lines[i:i + 3]
