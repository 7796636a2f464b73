"""The distillation kernels that are built are those that its choice by mode and row length
can start: a row part in shared memory is the loss and gradient's alone."""
import re
import shutil
import subprocess

import pytest

from moe_routing_capacity_gb300 import abi

from test_block_host import built_library  # noqa: F401

FORWARD, STEP, BACKWARD = 0, 1, 2


def test_no_kernel_without_a_caller():
    nm = shutil.which("nm")
    if not nm:
        pytest.skip("no nm")
    names = subprocess.run([nm, "-C", abi.LIB_PATH], capture_output=True, text=True, check=True).stdout
    pattern = r"distill_kernel<(float|unsigned short), (\d+), (\d+), (\d+), (\d+), \d+>"
    built = {(m[0], *map(int, m[1:])) for m in re.findall(pattern, names)}
    if not built:
        pytest.skip("a library without its local names")
    want = set()
    for z in ("float", "unsigned short"):
        for mode in (FORWARD, STEP, BACKWARD):       # threads a row, mode, vectors held, vectors in shared memory
            want |= {(z, 32, mode, 4, 0), (z, 32, mode, 0, 0), (z, 128, mode, 0, 0), (z, 256, mode, 0, 0)}
            want |= {(z, 480, mode, 0, 4), (z, 512, mode, 0, 8)} if mode == STEP else {(z, 512, mode, 0, 0)}
    assert built == want
