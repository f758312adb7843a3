"""Wait states around the copies into LDS, read off the built library (host only).

A copy into LDS takes its LDS address from m0 and its source's base from scalar registers.  The
hardware does not hold such an instruction back: it needs one wait state after a scalar write of m0,
and five after a vector instruction that wrote one of its scalar registers (v_readfirstlane, a
comparison).  The compiler keeps both distances for its own instructions, not inside an asm
statement or across its edge."""
import glob
import os
import re
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
M0, BASE = 1, 5


def _scalars(operands):
    """Scalar registers named in an operand list."""
    out = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", operands):
        out |= set(range(int(a), int(b) + 1))
    return out | {int(a) for a in re.findall(r"\bs(\d+)\b", operands)}


def _short(lines):
    """(function, instruction, what) of every copy into LDS that is too near to a write of its registers."""
    found, copies, function, before = [], 0, "", []
    for line in lines:
        m = re.match(r"(?:[0-9a-f]+ )?<(.*)>:", line)
        if m:
            function = m.group(1)
            continue
        text = line.split("//")[0].strip()
        if not text or not re.match(r"[a-z]+_", text):
            continue
        name, _, operands = text.partition(" ")
        if "load_lds" in name:
            copies += 1
            reads, states = _scalars(operands), 0
            for p in reversed(before[-BASE:]):
                pname, _, pops = p.partition(" ")
                target = pops.split(",")[0].strip()
                if target == "m0" and states < M0:
                    found.append((function, text, f"{states} wait states after {p}"))
                if pname.startswith("v_") and states < BASE and _scalars(target) & reads:
                    found.append((function, text, f"{states} wait states after {p}"))
                states += int(pops) + 1 if pname == "s_nop" else 1
        before.append(text)
    return found, copies


def test_the_reader_finds_both_kinds():
    near = ["<f>:", "v_readfirstlane_b32 s6, v10", "s_mov_b32 m0, s24", "global_load_lds_dwordx4 v7, s[6:7]"]
    assert len(_short(near)[0]) == 2
    apart = ["<f>:", "v_readfirstlane_b32 s6, v10", "s_mov_b32 m0, s24", "s_nop 3", "global_load_lds_dwordx4 v7, s[6:7]"]
    assert _short(apart) == ([], 1)
    apart[3] = "s_nop 2"
    assert len(_short(apart)[0]) == 1


def test_copies_into_lds_keep_their_distance(tmp_path):
    from post_weight_quantization_05_amd import _lib, build
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    here = tmp_path / "libqz.so"
    here.symlink_to(_lib.LIB_PATH)
    subprocess.run([OBJDUMP, "--offloading", str(here)], cwd=tmp_path, capture_output=True, check=True, timeout=100)
    found, copies, writes = [], 0, 0
    for code in sorted(glob.glob(str(tmp_path / "*gfx950"))):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", code], capture_output=True,
                              text=True, check=True, timeout=100).stdout
        if "load_lds" in text:
            f, c = _short(text.splitlines())
            found += f
            copies += c
            writes += len(re.findall(r"^\s*\w+ m0,", text, re.M))
    assert copies > 100     # the tile products' and the Hessian's
    assert not found, f"{len(found)} of {copies}: {found[:4]}"
    assert writes == copies     # the compiler keeps nothing of its own in m0 there
