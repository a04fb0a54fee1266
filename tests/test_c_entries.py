"""No C++ exception leaves a C entry point (CPU tests): it would end the caller's process."""
import subprocess
import sys

import pytest

from prefill_phase_attention_gb300 import build

# A process of its own, of bounded address space: the strict check copies the metadata of 2^28
# sequences to the host (3 GiB), which does not fit.
PROGRAM = """
import ctypes, resource, sys
lib = ctypes.CDLL(sys.argv[1])
lib.prefill_attn_last_error.restype = ctypes.c_char_p
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (256 << 20),) * 2)
P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
lib.prefill_attn_varlen_validate.argtypes = [P] * 10 + [I] * 6 + [F, I, P]
# cu_seqlens and the offsets apart from the tensors; nothing of them is read before the copies are allocated
got = lib.prefill_attn_varlen_validate(1 << 40, 2 << 40, 3 << 40, 4 << 40, 5 << 40, 6 << 40, 7 << 40, 8 << 40, 9 << 40,
                                       None, 1 << 28, 4, 1, 1, 1, 64, 0.125, 1, None)
print(got, lib.prefill_attn_last_error().decode())
"""


@pytest.fixture(scope="module")
def library():
    return build.build()


def test_out_of_host_memory_is_a_status(library):
    r = subprocess.run([sys.executable, "-c", PROGRAM, library], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, f"the process ended with {r.returncode}: {r.stderr[-300:]}"
    assert r.stdout.split()[0] == "3" and "host memory" in r.stdout, r.stdout
