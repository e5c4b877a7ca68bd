"""How many waves of each ring kernel a SIMD holds, by the registers that the
library's code asks for.  A ring launch needs all its workgroups resident at
once, so a kernel that takes more registers refuses launches that it took.  No
GPU needed."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from ring_all_reduce_channelmask_amd import _lib

TOOLS = "/opt/rocm/llvm/bin"
REGISTERS = 512  # of a lane, on a SIMD of gfx950; a wave has a multiple of 8
LL, LL128, SIMPLE = 0, 1, 2


@pytest.mark.skipif(not os.path.exists(f"{TOOLS}/llvm-readelf"), reason="needs llvm-readelf")
def test_waves_of_the_ring_kernels(tmp_path):
    lib = shutil.copy(_lib.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([f"{TOOLS}/llvm-objdump", "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    waves = {}
    for part in glob.glob(str(tmp_path / "*gfx950*")):
        notes = subprocess.run([f"{TOOLS}/llvm-readelf", "--notes", part], check=True, capture_output=True, text=True).stdout
        for name, count in re.findall(r"\.name:\s+(\S*ring_allreduce_kernel\S*).*?\.vgpr_count:\s+(\d+)", notes, re.S):
            # the payload type with its operator, then the protocol
            payload, op, proto = re.search(r"Ty(I32|F32|BF16)ILi(\d)EEELi(\d)E", name).groups()
            waves[payload, int(op), int(proto)] = REGISTERS // (-(-int(count) // 8) * 8)
    assert len(waves) == 3 * 6 * 3
    for (payload, op, proto), n in waves.items():
        assert n >= (2 if proto == SIMPLE and payload != "BF16" else 3), (payload, op, proto, n)
