"""The 8-bit product's kernels on emulated workgroups (tests/emulate), on the CPU:
csrc/fsdp_fp8_tiles.h and fsdp_fp8_matmul.hip as they are, with lanes as fibers and
loads into LDS that land as late as the kernel's own waits allow, at once, or at
random.  A wait that leaves a load on its way, a stage that is overwritten while a
wave still reads it, a read behind an operand and a byte written beside the result
each fail.  The products are of whole numbers and compared exactly.
"""
import concurrent.futures
import os
import shutil

import pytest

from test_sanitizers import CSRC, HIPCC, ROOT, _run, pytestmark  # noqa: F401

EMULATE = os.path.join(ROOT, "tests", "emulate")
FROM_CSRC = ["fsdp_fp8_tiles.h", "fsdp_fp8_matmul.hip", "fsdp_fp8.h", "fsdp_kernels.h"]
PARTS = 4


@pytest.fixture(scope="module")
def products(tmp_path_factory):
    """The program, built from copies: a source's includes are looked for beside it first."""
    d = str(tmp_path_factory.mktemp("emulate"))
    for f in [os.path.join(CSRC, f) for f in FROM_CSRC] + [os.path.join(EMULATE, f) for f in os.listdir(EMULATE)]:
        shutil.copy(f, d)
    exe = os.path.join(d, "products")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(HIPCC)))
    _run([HIPCC, "-x", "c++", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I", d,
          "-I", os.path.join(ROOT, "include"), "-std=c++17", "-O2", "-ffp-contract=off", "-w",
          os.path.join(d, "products.cpp"), "-o", exe])
    return exe


def test_products_on_emulated_workgroups(products):
    with concurrent.futures.ThreadPoolExecutor(PARTS) as ex:
        for r in ex.map(lambda i: _run([products, str(i), str(PARTS)]), range(PARTS)):
            assert "products done" in r.stdout
