"""The library's own kernels as they were compiled: instructions that gfx950 has been seen to get wrong."""
import os
import re
import shutil
import subprocess

import pytest

from gated_deltanet_linear_step_amd import ops

LLVM = "/opt/rocm/llvm/bin"
TOOLS = [os.path.join(LLVM, n) for n in ("llvm-objdump", "llvm-readelf")]
SHIFT = re.compile(r"\bv_(?:lshlrev_b64|lshrrev_b64|ashrrev_i64)(?:_e64)?\s+v\[\d+:\d+\], v(\d+),")


def kernels(path, where):
    """(name, VGPRs that a wave is allotted, lines of code) of every kernel of the library."""
    lib = shutil.copy(path, where / "lib.so")
    subprocess.run([TOOLS[0], "--offloading", lib], cwd=where, check=True, capture_output=True)
    for part in sorted(where.glob("lib.so.*gfx950")):
        notes = subprocess.run([TOOLS[1], "--notes", part], check=True, capture_output=True, text=True).stdout
        count = {}
        for name, rest in re.findall(r"\.name:\s+(_Z\S+)\n(.*?)(?=\.name:\s+_Z|\Z)", notes, re.S):
            count[name] = int(re.search(r"\.vgpr_count:\s+(\d+)", rest).group(1))
        name, lines = None, []
        text = subprocess.run([TOOLS[0], "-d", "--no-show-raw-insn", part], check=True, capture_output=True, text=True).stdout
        for line in text.splitlines() + ["0 <>:"]:
            start = re.match(r"[0-9a-f]+ <(\S*)>:", line)
            if not start:
                lines.append(line)
                continue
            if name in count:
                yield name, (count[name] + 7) // 8 * 8, lines
            name, lines = start.group(1), []


@pytest.mark.skipif(not all(os.path.exists(t) for t in TOOLS), reason="needs ROCm's LLVM tools")
def test_no_64_bit_shift_takes_its_amount_from_the_last_register(tmp_path):
    """csrc/gdn_attn_device.h says what that did."""
    ops.load()
    seen, wrong = 0, []
    for name, allotted, lines in kernels(ops.LIB_PATH, tmp_path):
        seen += 1
        wrong += [(name, line.strip()) for line in lines for m in [SHIFT.search(line)] if m and int(m.group(1)) == allotted - 1]
    assert seen > 300, "the library's kernels were not found"
    assert not wrong, wrong
