"""No store of 12 or 16 bytes takes its place from a scalar offset, in the machine code
of the built libraries.

Such a store reads its data's registers after it has been issued.  The compiler
keeps the next instruction from writing them, but not where the store has a scalar
offset register; on gfx950 the first register's last lanes were then sent with the
next value now and then.  Kernels put the place into the buffer resource or the
vector offset.
"""

import os
import re
import shutil
import subprocess

import pytest

from test_i8_tile_wait import OBJDUMP, ROOT

STORE = re.compile(r"buffer_store_dwordx[34] \S+, (?:off|v\d+), s\[\d+:\d+\], (s\d+|vcc_\w+|ttmp\d+|m0)\b")


def test_the_pattern():
    assert STORE.search("buffer_store_dwordx4 v[2:5], v44, s[24:27], s14 offen nt")
    assert STORE.search("buffer_store_dwordx3 v[2:4], off, s[24:27], s14")
    assert not STORE.search("buffer_store_dwordx4 v[2:5], v44, s[24:27], 0 offen nt")
    assert not STORE.search("buffer_store_dwordx2 v[2:3], v44, s[24:27], s14 offen nt")


@pytest.mark.parametrize("lib", ["libfp8q.so", "libfp8q_debug.so"])
def test_no_wide_store_with_a_scalar_offset(lib, tmp_path):
    so = shutil.copy(os.path.join(ROOT, "fine_grained_block_fp8q_amd", lib), tmp_path)
    subprocess.run([OBJDUMP, "--offloading", so], cwd=tmp_path, check=True, stdout=subprocess.DEVNULL)
    code = [f for f in sorted(os.listdir(tmp_path)) if "gfx950" in f]
    assert code
    stores = 0
    for f in code:
        text = subprocess.run([OBJDUMP, "-d", f], cwd=tmp_path, check=True, capture_output=True,
                              text=True).stdout
        bad = [l for l in text.splitlines() if STORE.search(l)]
        assert not bad, bad[:3]
        stores += text.count("buffer_store_dwordx4")
    assert stores > 0
