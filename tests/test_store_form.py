"""The form of the library's wide stores, from its own gfx950 code: a buffer
store of 12 or 16 bytes takes its row's offset from the lanes.  With one in a
scalar register nothing keeps the next instruction from overwriting the
registers that are being stored, and what they became has been stored (four
lanes of sixteen, now and then); without one the compiler waits."""
import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

from sparse_tiled_gemm_amd import gemm as G

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WIDE = re.compile(r"\bbuffer_store_(?:dwordx[34]|(?:format_)?xyzw?)\s+(\S+), (\S+), (s\[\d+:\d+\]), (\S+)")


def wide_stores(code):
    """(a wide store's kernel, its scalar offset) of a code object."""
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", code], capture_output=True, text=True,
                          check=True).stdout
    found, kernel = [], None
    for line in text.splitlines():
        if line.endswith(">:"):
            kernel = line.split("<", 1)[1][:-2]
        elif m := WIDE.search(line):
            found.append((kernel, m.group(4)))
    return found


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump here")
def test_wide_stores_take_no_scalar_offset(tmp_path):
    lib = shutil.copy(G.LIB_PATH, tmp_path / "lib.so")  # (the parts are put beside it)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], capture_output=True, check=True)
    parts = [str(p) for p in tmp_path.iterdir() if p.name.endswith("gfx950")]
    assert parts
    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        stores = [s for found in ex.map(wide_stores, parts) for s in found]
    assert len(stores) > 100  # (the epilogues' among them: the text was understood)
    bad = sorted({kernel for kernel, offset in stores if not offset.isdigit()})
    assert not bad, "%d of %d wide stores: %s" % (
        sum(not o.isdigit() for _, o in stores), len(stores), bad[:3])
