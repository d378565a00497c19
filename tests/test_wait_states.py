"""Wait states around the loads that are written out in inline assembly.

The compiler's hazard pass does not look into an asm block, so what the
CDNA ISA asks for between instructions has to be kept by hand there.  The
library's own gfx950 code is disassembled, and every global load to LDS is
looked at, instruction by instruction within its basic block:

  M0        a scalar write of M0 needs one wait state before a load to LDS
            that uses it
  scalars   a scalar register that a vector instruction wrote needs five
            before a vector memory instruction reads it (its base address)
"""
import os
import re
import shutil
import subprocess

import pytest

import bit_exact_matrix_amd as mm

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def registers(text):
    """Scalar registers named in an operand: s7, s[4:7], vcc, m0."""
    out = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out.update(range(int(a), int(b) + 1))
    out.update(int(a) for a in re.findall(r"\bs(\d+)\b", text))
    if re.search(r"\bvcc\b", text):
        out.add("vcc")
    if re.search(r"\bm0\b", text):
        out.add("m0")
    return out


def faults(lines):
    """(kernel, load, reason) of every load to LDS that comes too early, and
    the number of loads looked at."""
    bad, loads, kernel = [], 0, None
    recent = []  # (wait states since, registers, by the vector unit), newest last
    for line in lines:
        head = re.match(r"^[0-9a-f]+ <(.+)>:", line)
        if head:
            kernel, recent = head.group(1), []
            continue
        line = line.split("//")[0].strip()
        parts = line.split(None, 1)
        if not parts or not re.match(r"[a-z]+_", parts[0]):
            continue
        op, args = parts[0], parts[1] if len(parts) > 1 else ""
        if op.startswith("global_load_lds"):
            loads += 1
            read = registers(args)
            for age, regs, vector in recent:
                if not vector and "m0" in regs and age < 1:
                    bad.append((kernel, line, "M0 written just before"))
                if vector and regs & read and age < 5:
                    bad.append((kernel, line, f"scalar base written {age} wait states before"))
        states = int(args, 0) + 1 if op == "s_nop" else 1
        recent = [(age + states, regs, vector) for age, regs, vector in recent
                  if age + states < 5]
        dest = args.split(",")[0]
        if op.startswith("v_cmp") and not op.startswith("v_cmpx"):
            recent.append((0, registers(dest) or {"vcc"}, True))
        elif op.startswith("v_"):
            # the destination, and a carry's
            regs = registers(dest)
            if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[iu]64", op):
                regs |= registers(args.split(",")[1])
            if regs:
                recent.append((0, regs, True))
        elif op.startswith("s_") and "m0" in registers(dest):
            recent.append((0, {"m0"}, False))
    return bad, loads


def test_the_check_itself():
    """It sees a missing wait, and is content with the states in place."""
    text = """
0000000000000000 <k>:
  s_mov_b32 m0, s3
  global_load_lds_dwordx4 v1, s[4:5]
  v_readfirstlane_b32 s4, v9
  s_mov_b32 m0, s3
  s_nop 0
  global_load_lds_dwordx4 v1, s[4:5]
  v_readfirstlane_b32 s4, v9
  s_mov_b32 m0, s3
  s_nop 3
  global_load_lds_dwordx4 v1, s[4:5]
  v_cmp_gt_u32_e64 s[4:5], v1, v2
  v_readfirstlane_b32 s6, v9
  s_mov_b32 m0, s6
  s_nop 0
  global_load_lds_dwordx4 v[1:2], off
"""
    bad, loads = faults(text.splitlines())
    assert loads == 4
    assert [b[2] for b in bad] == ["M0 written just before",
                                   "scalar base written 2 wait states before"]


def test_loads_to_lds_keep_their_wait_states(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    lib = shutil.copy(mm.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", str(lib)], cwd=tmp_path, check=True,
                   capture_output=True)
    bad, loads = [], 0
    for name in sorted(os.listdir(tmp_path)):
        if not name.endswith("gfx950"):
            continue
        with subprocess.Popen([OBJDUMP, "-d", "--no-show-raw-insn", str(tmp_path / name)],
                              stdout=subprocess.PIPE, text=True) as p:
            b, n = faults(p.stdout)
        bad += b
        loads += n
    assert loads > 1000, "the kernels' direct loads"
    kinds = {(k, r) for k, _, r in bad}
    assert not bad, f"{len(bad)} of {loads} loads: " + "; ".join(
        f"{k}: {r}" for k, r in sorted(kinds)[:8])
