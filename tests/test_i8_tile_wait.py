"""The wait between the last matrix product of an int8 tile and the first use of
its sums, in the machine code of the built libraries.

The products are inline asm, so the compiler inserts no wait of its own for their
results: the kernel has to, and every use of an accumulation register must come
after it.
"""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc"))),
                       "llvm", "bin", "llvm-objdump")
PRODUCT = "v_mfma_i32_16x16x64_i8"
# An 8-pass product's result may be read by the vector ALU 11 states after it, a
# 16-pass one's 19 after it.
STATES = 19


def _i8_kernels(lib, tmp):
    """{kernel: [(offset in the kernel, instruction, offset branched to or None)]}."""
    so = shutil.copy(lib, tmp)
    subprocess.run([OBJDUMP, "--offloading", so], cwd=tmp, check=True, stdout=subprocess.DEVNULL)
    kernels = {}
    for f in sorted(os.listdir(tmp)):
        if "gfx950" not in f:
            continue
        text = subprocess.run([OBJDUMP, "-d", f], cwd=tmp, check=True, capture_output=True,
                              text=True).stdout
        name, start = None, 0
        for line in text.splitlines():
            m = re.match(r"([0-9a-f]+) <(\S+)>:", line)
            if m:
                start, name = int(m.group(1), 16), m.group(2)
                continue
            m = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+):(.*)", line)
            if m and name and "i8_tile_kernel" in name:
                to = re.search(r"<\S+\+0x([0-9a-f]+)>", m.group(3))
                kernels.setdefault(name, []).append((int(m.group(2), 16) - start, m.group(1),
                                                     int(to.group(1), 16) if to else None))
    return kernels


def _after_the_loop(code):
    """The instructions that run after the last product's block, when the loop is left."""
    at = {off: i for i, (off, _, _) in enumerate(code)}
    i = max(i for i, c in enumerate(code) if c[1].startswith(PRODUCT)) + 1
    while i < len(code):
        _, text, to = code[i]
        yield text
        i = at[to] if text.startswith("s_branch") else i + 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
@pytest.mark.parametrize("lib", ["libfp8q.so", "libfp8q_debug.so"])
def test_sums_are_used_after_the_wait(lib, tmp_path):
    kernels = _i8_kernels(os.path.join(ROOT, "fine_grained_block_fp8q_amd", lib), tmp_path)
    assert len(kernels) == 20           # five tiles, gated or not, two output types
    for name, code in kernels.items():
        states, use = 0, None
        for c in _after_the_loop(code):
            if re.search(r"\ba(\d+|\[\d+:\d+\])", c):
                use = c
                break
            m = re.match(r"s_nop (\d+)", c)
            if m:
                states += int(m.group(1)) + 1
        assert use, f"{name}: no use of the sums found"
        assert states >= STATES, f"{name}: `{use}` after {states} waited states"
