"""The built products that are cut along k hand partial tiles from workgroup to
workgroup: every wave has to wait for its own stores before the barrier that lets
one thread announce them.  A missing wait shows now and then at most, so it is
looked for in the machine code of the library built here.  CPU only."""

from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sharded_mixed_precision_zero_amd", "libzeroshard.so")
OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")


def _kernels(tmp_path):
    """(name, instructions) of each kernel in the library."""
    lib = shutil.copy(LIB, tmp_path)  # the code objects are written beside it
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, timeout=60)
    out = []
    for part in sorted(os.listdir(tmp_path)):
        if not part.endswith("gfx950"):
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-leading-addr", "--no-show-raw-insn",
                               os.path.join(tmp_path, part)], check=True, capture_output=True,
                              text=True, timeout=120).stdout
        for block in re.split(r"^<", text, flags=re.M)[1:]:
            name, _, body = block.partition(">:")
            out.append((name, [line.split("//")[0].strip() for line in body.splitlines()]))
    return out


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_every_wave_waits_for_its_stores_before_the_handover(tmp_path):
    found = 0
    for name, code in _kernels(tmp_path):
        for at, line in enumerate(code):
            if not line.startswith("buffer_wbl2"):
                continue
            found += 1
            barrier = max(i for i in range(at) if code[i] == "s_barrier")
            store = max(i for i in range(barrier) if code[i].startswith("global_store"))
            waits = [w for w in code[store:barrier] if w.startswith("s_waitcnt")]
            assert any("vmcnt(0)" in w for w in waits), (name, code[store:at + 1])
    # four kinds of product in three tile shapes each are cut
    assert found == 12, found
