"""A kernel is found by its name: what the host registers has to be what the
device code is called.  The two are compiled apart, and count unnamed types in
a signature apart; a launch of a kernel whose names differ ends the process."""
import os
import re
import shutil
import subprocess

import pytest

import bit_exact_matrix_amd as mm

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def symbols(path):
    out = subprocess.run([OBJDUMP, "-t", str(path)], check=True, capture_output=True, text=True)
    return {line.split()[-1] for line in out.stdout.splitlines() if re.match(r"^[0-9a-f]{8}", line)}


def test_every_kernel_has_one_name(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    lib = shutil.copy(mm.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", str(lib)], cwd=tmp_path, check=True,
                   capture_output=True)
    device = set()
    for name in os.listdir(tmp_path):
        if name.endswith("gfx950"):
            device |= {s[:-3] for s in symbols(tmp_path / name) if s.endswith(".kd")}
    assert len(device) > 100
    missing = device - symbols(lib)
    assert not missing, sorted(missing)[:5]
