"""The compiled kernels, read instruction by instruction: no 64-bit vector shift
takes its amount from the last vector register that its wave is given.

Measured on MI355X: such a shift takes another amount as soon as a second wave
lives on the same SIMD, as if the amount's register were the lower one of a pair
whose upper one lies behind the wave's own.  A product of 16x16384x123 had up to
24578 wrong values with 40 registers a wave and the amount in the 40th, and none
with the same instructions and 48.  The compiler does not avoid it, so
shifts by a variable amount are written in 32 bits where that is possible, and
the library is looked through here.  Needs the built library and LLVM's tools."""
import os
import re
import struct
import subprocess

import pytest

from gradient_compression_distributed_lc_amd import build, tlc

LLVM = "/opt/rocm/llvm/bin"
SHIFT = re.compile(r"\sv_(?:lshlrev_b64|lshrrev_b64|ashrrev_i64)(?:_e64)? v\[\d+:\d+\], v(\d+),")


def code_objects(data):
    """The gfx950 code objects in a library's bytes."""
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(magic))
        p = at + len(magic) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            p += 24 + length
            if b"gfx950" in data[p - length:p]:
                yield data[at + offset:at + offset + size]
        at = data.find(magic, p)


def shifts_by_the_last_register(assembly, registers):
    """(kernel, instruction) of each; registers: how many each kernel's waves are given, in eights."""
    kernel, found = None, []
    for line in assembly.splitlines():
        m = re.match(r"[0-9a-f]+ <(\S+)>:", line)
        if m:
            kernel = m[1]
        m = SHIFT.search(line)
        if m and int(m[1]) + 1 == -(-registers[kernel] // 8) * 8:
            found.append((kernel, line.split("//")[0].strip()))
    return found


def test_the_rule_itself():
    text = "0000 <k>:\n\tv_lshrrev_b64 v[16:17], v39, v[18:19]  // 00\n\tv_lshlrev_b64 v[2:3], v38, v[4:5]\n" \
           "\tv_lshlrev_b64 v[2:3], 1, v[4:5]\n\tv_ashrrev_i64 v[2:3], v31, v[4:5]\n"
    assert shifts_by_the_last_register(text, {"k": 40}) == [("k", "v_lshrrev_b64 v[16:17], v39, v[18:19]")]
    assert len(shifts_by_the_last_register(text, {"k": 35})) == 1 and not shifts_by_the_last_register(text, {"k": 41})
    assert shifts_by_the_last_register(text, {"k": 32}) == [("k", "v_ashrrev_i64 v[2:3], v31, v[4:5]")]


def test_no_shift_by_a_waves_last_register(tmp_path):
    if not os.path.exists(os.path.join(LLVM, "llvm-objdump")):
        pytest.skip("LLVM's tools are not installed")
    tlc.lib()
    with open(build.LIB, "rb") as f:
        objects = list(code_objects(f.read()))
    assert len(objects) == len(build.SOURCES)
    kernels, found = 0, []
    for k, data in enumerate(objects):
        path = tmp_path / f"{k}.co"
        path.write_bytes(data)
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", str(path)], check=True,
                               capture_output=True, text=True).stdout
        registers = {m[1]: int(m[2]) for m in
                     re.finditer(r"\.name:\s+(\S+)\n(?:(?!\.name:).)*?\.vgpr_count:\s+(\d+)", notes, re.S)}
        registers = {name: n for name, n in registers.items() if name.startswith("_Z")}
        text = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--mcpu=gfx950", str(path)], check=True,
                              capture_output=True, text=True).stdout
        kernels += len(registers)
        found += shifts_by_the_last_register(text, registers)
    assert kernels > 200
    assert not found, found
