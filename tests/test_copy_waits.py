"""Wait states before the copies to LDS in the library as compiled.

The copies (global_load_lds) are inline assembly, for which the compiler inserts no wait states.  They read M0 and, in one
form, a base address in scalar registers: one wait state after a scalar instruction that writes M0 (the compiler puts one
before its own copies), five after a vector instruction that writes a scalar register they read.  Every instruction between is
one; s_nop n is n + 1.
"""

import os
import re
import struct
import subprocess

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "quantized_linear_moe_amd", "libqe.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(blob):
    """The gfx950 code objects of the bundles in a library (little-endian: count, then offset, size and name of each)."""
    at = blob.find(MAGIC)
    while at >= 0:
        p = at + len(MAGIC)
        (count,) = struct.unpack_from("<Q", blob, p)
        p += 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", blob, p)
            name = blob[p + 24:p + 24 + n]
            p += 24 + n
            if name.endswith(b"gfx950") and size:
                yield blob[at + offset:at + offset + size]
        at = blob.find(MAGIC, at + 1)


def _scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {operand} if re.fullmatch(r"s\d+|m0", operand) else set()


def _short_waits(lines):
    """Copies and those of them that follow a write too closely."""
    copies, short = 0, []
    for i, line in enumerate(lines):
        if not line.startswith("global_load_lds"):
            continue
        copies += 1
        reads = {"m0"}.union(*[_scalars(o.strip(",")) for o in line.split()[1:]])
        states = 0
        for before in reversed(lines[max(0, i - 5):i]):
            op, *rest = before.split()
            if op == "s_nop":
                states += int(rest[0], 0) + 1
                continue
            written = _scalars(rest[0].strip(",")) & reads if rest else set()
            if written and (op.startswith("v_") and states < 5 or "m0" in written and states < 1):
                short.append((before, line))
            states += 1
    return copies, short


def test_the_scan_finds_short_waits():
    """The scan itself, on lines made up for it."""
    copy = "global_load_lds_dwordx4 v1, s[4:5]"
    for lines, bad in ((["s_mov_b32 m0, s1", copy], 1), (["s_mov_b32 m0, s1", "s_nop 0", copy], 0),
                       (["s_add_i32 m0, s1, 0x400", "v_mov_b32_e32 v1, v2", copy], 0),
                       (["s_add_u32 s4, s1, s2", "s_nop 0", copy], 0),
                       (["v_readfirstlane_b32 s5, v2", "s_nop 3", copy], 1), (["v_readlane_b32 s4, v2, 1", "s_nop 4", copy], 0),
                       (["v_readfirstlane_b32 m0, v2", "s_nop 0", copy], 1), (["v_readfirstlane_b32 s9, v2", copy], 0)):
        assert _short_waits(lines) == (1, [(lines[0], copy)] if bad else []), lines


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs ROCm's llvm-objdump")
def test_copies_wait_for_what_they_read(tmp_path):
    with open(LIB, "rb") as f:
        objects = list(_code_objects(f.read()))
    assert objects
    copies = 0
    for n, code in enumerate(objects):
        path = tmp_path / f"{n}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", "--no-show-raw-insn", str(path)], check=True,
                              capture_output=True, text=True).stdout
        lines = [m[1].strip() for m in re.finditer(r"^\t(.*?)(?:\s*//.*)?$", text, re.M)]
        some, short = _short_waits(lines)
        copies += some
        assert not short, f"{len(short)} of {some}, the first: {short[0]}"
    assert copies > 0
