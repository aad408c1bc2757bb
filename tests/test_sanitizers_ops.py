"""The host layer of the gradient norm, clipping and the 4-bit microscaled
blocks under AddressSanitizer + UndefinedBehaviorSanitizer and under
ThreadSanitizer on the CPU (no GPU): tests/sanitize/ops_checks.cpp drives every
entry point over validation, tables and launch planning with never-dereferenced
device pointers, sizes up to the ends of int64 among them.  Any sanitizer report
fails the run.
"""
import concurrent.futures
import os

import pytest

from test_sanitizers import COMMON, CSRC, HERE, HIPCC, HOST_ASAN_UBSAN, HOST_TSAN, _run, pytestmark  # noqa: F401

SOURCES = ["fsdp_kernels.hip", "fsdp_abi.cpp", "fsdp_norm.hip", "fsdp_norm_abi.cpp", "fsdp_mx4.hip",
           "fsdp_mx4_matmul.hip", "fsdp_mx4_few.hip", "fsdp_mx4_abi.cpp"]


@pytest.mark.parametrize("tag,san", [("asan", HOST_ASAN_UBSAN), ("tsan", HOST_TSAN)])
def test_host_layer_of_the_operators(tmp_path, tag, san):
    srcs = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(HERE, "ops_checks.cpp")]
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]
    jobs = min(len(srcs), int(os.environ.get("MAX_JOBS", "0")) or (os.cpu_count() or 4), 16)
    with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
        list(ex.map(lambda so: _run([HIPCC] + COMMON + san + ["-x", "hip", "-c", so[0], "-o", so[1]]),
                    zip(srcs, objs)))
    exe = str(tmp_path / "ops_checks")
    _run([HIPCC, "--offload-arch=gfx950"] + san + objs + ["-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", HIP_VISIBLE_DEVICES="",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", TSAN_OPTIONS="halt_on_error=1:second_deadlock_stack=1")
    assert "ops sanitizer checks" in _run([exe], env=env).stdout
