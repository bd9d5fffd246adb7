"""The library's own machine code: no vector register is written between the place where a skipped branch comes back and
the instruction that gives all lanes back there.  A register allocator under pressure has put moves there (of a value that
every lane needs later, out of the way of others): the lanes that did not take the branch then go on with what the other
register held before, an address out of range among the outcomes.  (CPU; reads liblconv.so, which is built here.)"""
import os
import re
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "fft_long_convolution_amd", "liblconv.so")


def code_objects(path):
    """The gfx950 code objects in the library's bundles."""
    data = open(path, "rb").read()
    for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data):
        count, = struct.unpack_from("<Q", data, m.start() + 24)
        at = m.start() + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + length]
            at += 24 + length
            if size and b"gfx950" in name:
                yield data[m.start() + offset:m.start() + offset + size]


def copies_under_a_partial_mask(text):
    """(kernel, address, instruction) of vector writes between the target of an s_cbranch_execz and `s_or_b64 exec, exec`."""
    found, kernel, code = [], None, []

    def kernel_done():
        targets = set()
        for pc, op, _, line in code:
            m = op == "s_cbranch_execz" and re.search(r"\+0x([0-9a-f]+)>", line)
            if m:
                targets.add(int(m.group(1), 16))
        start = code[0][0] if code else 0
        pending = None
        for pc, op, args, _ in code:
            if pc - start in targets:
                pending = []
            if pending is None:
                continue
            if op == "s_or_b64" and args.startswith("exec, exec"):
                found.extend((kernel, hex(p), i) for p, i in pending)
                pending = None
            elif op.startswith(("s_cbranch", "s_branch", "s_endpgm")) or "saveexec" in op or args.startswith("exec"):
                pending = None
            elif op.startswith("scratch_") or (op.startswith("v_") and not op.startswith(("v_cmp", "v_readlane", "v_readfirstlane", "v_writelane"))):
                pending.append((pc, op + " " + args))

    for line in text.splitlines():
        m = re.match(r"[0-9a-f]+ <(\w+)>:", line)
        if m:
            kernel_done()
            kernel, code = m.group(1), []
            continue
        m = re.match(r"\s+([a-z]\w+)\s*(.*?)\s*// ([0-9A-F]+):(.*)", line)
        if m:
            code.append((int(m.group(3), 16), m.group(1), m.group(2), line))
    kernel_done()
    return found


def test_the_scan_sees_such_a_copy():
    text = """
0000000000001000 <planted>:
\ts_and_saveexec_b64 s[8:9], vcc                   // 000000001000: BE882002
\ts_cbranch_execz 2                                // 000000001004: BF8800A2 <planted+0x10>
\tglobal_load_dwordx4 v[0:3], v[2:3], off          // 000000001008: DC5C8000 007F0002
\tv_accvgpr_write_b32 a176, v14                    // 000000001010: D3D940B0 1800010E
\ts_or_b64 exec, exec, s[8:9]                      // 000000001018: 87FE087E
"""
    assert copies_under_a_partial_mask(text) == [("planted", "0x1010", "v_accvgpr_write_b32 a176, v14")]
    inside = text.replace("<planted+0x10>", "<planted+0x18>")     # the same move before the branch comes back is the branch's own
    assert copies_under_a_partial_mask(inside) == []


def test_no_register_is_moved_under_a_partial_mask(tmp_path):
    tool = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(LIB) or not os.path.exists(tool):
        pytest.skip("no built library, or no llvm-objdump")
    found, kernels = [], 0
    for i, elf in enumerate(code_objects(LIB)):
        path = tmp_path / f"{i}.elf"
        path.write_bytes(elf)
        r = subprocess.run([tool, "-d", str(path)], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
        assert r.returncode == 0, r.stderr[-500:]
        kernels += len(re.findall(r"^[0-9a-f]+ <\w+>:", r.stdout, flags=re.M))
        found += copies_under_a_partial_mask(r.stdout)
    assert kernels > 100
    assert not found, found[:5]
