"""What the layer norm, the short causal convolution and the selective scan ask of the CUDA
runtime, with a stand-in for the runtime that notes each call and launches nothing: a kernel's
limit of shared memory does not depend on the call (it is the function's, shared by all
threads), and a failed question to the runtime is that call's own.  On the CPU, in processes
of their own."""
import json
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = r"""
#include <stdio.h>
#include <stdlib.h>
typedef struct { unsigned x, y, z; } dim3;
typedef struct { dim3 grid, block; size_t shared; void* stream; void* attrs; unsigned n; } config;
static int device, failures;
void fake_device(int d) { device = d; }
void fake_failures(int n) { failures = n; }
int cudaGetDevice(int* d) { *d = device; return 0; }
int cudaGetLastError(void) { return 0; }
int cudaDeviceGetAttribute(int* v, int attr, int d) {
  *v = attr == 75 ? 10 : attr == 76 ? 3 : 152;   // compute capability, else SMs
  return 0;
}
int cudaFuncSetAttribute(const void* f, int attr, int v) {
  if (attr == 8) printf("[\"limit\", %zu, %d]\n", (size_t)f, v);
  return 0;
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int threads,
                                                           size_t shared, unsigned flags) {
  printf("[\"asked\", %zu]\n", (size_t)f);
  if (failures > 0) { --failures; *n = 77; return 999; }
  *n = device == 0 ? 6 : 2;
  return 0;
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int threads,
                                                  size_t shared) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(n, f, threads, shared, 0);
}
int cudaLaunchKernelExC(const config* c, const void* f, void** args) {
  printf("[\"launch\", %zu, %zu, %u]\n", (size_t)f, c->shared, c->grid.x);
  return 0;
}
int cudaMemsetAsync(void* p, int v, size_t n, void* st) { return 0; }
"""
CALLS = r"""
import ctypes, os, sys
lib = ctypes.CDLL(sys.argv[1])
fake = ctypes.CDLL(sys.argv[2])
P, I64, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
at = lambda n: P(n << 42)
def say(*what):
    fake.fflush(None)
    sys.stdout.write("[" + ", ".join('"%s"' % w if isinstance(w, str) else str(w) for w in what) + "]\n")
    sys.stdout.flush()
def norm_bwd(D, dtype=0, off=0):
    return lib.sanatan_layer_norm_bwd(at(1), None, at(2), at(3), at(4), dtype, I64(999), D,
                                      P((5 << 42) + 4 * off), at(6), at(7), at(8), SZ(1 << 40), None)
def conv_fwd(B, T, D, K=4, dtype=0):
    return lib.sanatan_causal_conv_fwd(at(1), I64(D), at(2), None, dtype, 1, None, B, T, D, K,
                                       None, at(3), None, None)
def conv_bwd(B, T, D, K=4, dtype=0):
    return lib.sanatan_causal_conv_bwd(at(1), I64(D), at(2), None, at(3), dtype, 1, None, B, T, D,
                                       K, None, None, at(4), at(5), None, None, at(6),
                                       SZ(1 << 40), None)
def scan(B, T, D, N, dtype=0):
    ld = (I64(D), at(4), I64(N), at(5), I64(N), at(6), None, None, dtype, 1, None, B, T, D, N)
    s = lib.sanatan_selective_scan_fwd(at(1), at(2), at(3), *ld, None, at(7), None, at(8), at(9),
                                       SZ(1 << 40), None)
    return s or lib.sanatan_selective_scan_bwd(
        at(1), at(2), at(3), *ld, at(7), at(8), None, at(10), at(11), at(12), at(13), at(14),
        at(15), None, None, None, at(9), SZ(1 << 40), None)
"""


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    """calls(code): what the runtime is asked and told by the library in a new process."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("needs gcc")
    from constant_state_recurrence_gb300 import build
    lib = build.build(quiet=True)
    where = tmp_path_factory.mktemp("runtime")
    (where / "fake.c").write_text(FAKE)
    fake = str(where / "fake.so")
    subprocess.run([gcc, "-shared", "-fPIC", "-O1", "-o", fake, str(where / "fake.c")], check=True)

    def run(code):
        r = subprocess.run([sys.executable, "-c", CALLS + code, lib, fake], capture_output=True,
                           text=True, timeout=120, env=dict(os.environ, LD_PRELOAD=fake), cwd=ROOT)
        assert r.returncode == 0, r.stderr
        return [json.loads(line) for line in r.stdout.splitlines()]
    return run


def test_a_kernels_limit_of_shared_memory_is_the_same_at_every_call(calls):
    """Two threads may set and launch in any order: a limit that follows the call's own size
    could be lowered between another call's two steps."""
    log = calls("""
for dtype in (0, 1):
    for off in (0, 1):
        for D in (5, 32, 768, 769, 1024, 1152, 1280, 2048, 2560, 4096, 5120, 8192, 20000):
            say("status", norm_bwd(D, dtype, off))
    for K in (1, 2, 3, 4, 7):
        for D in (64, 63, 1536):
            say("status", conv_fwd(2, 500, D, K, dtype)); say("status", conv_bwd(2, 500, D, K, dtype))
    for N in (1, 16, 20, 32, 40, 64, 100, 128):
        for D in (64, 63, 1536):
            for T in (20, 500):
                say("status", scan(2, T, D, N, dtype))
""")
    assert all(x[1] == 0 for x in log if x[0] == "status")
    assert len({x[1] for x in log if x[0] == "launch"}) > 40
    limits = {}
    for x in log:
        if x[0] == "limit":
            limits.setdefault(x[1], set()).add(x[2])
        elif x[0] == "launch" and x[2] > 48 * 1024:
            assert x[2] <= max(limits[x[1]])
    assert limits and all(len(sizes) == 1 for sizes in limits.values()), limits


def test_a_failed_question_is_the_calls_own(calls):
    """The convolution's run length comes from how many blocks the device holds: a call whose
    question fails returns an error and launches nothing, the next asks again, a device's answer
    is kept, and is not another device's."""
    one = "say('status', conv_fwd(8, 4096, 1536, 4, 1))\n"
    want = {}
    for device in (0, 1):
        log = calls(f"fake.fake_device({device})\n" + one)
        assert [x[0] for x in log] == ["asked", "launch", "status"] and log[2][1] == 0
        want[device] = log[1][3]
    assert want[0] != want[1]
    log = calls("fake.fake_failures(2)\n" + 4 * one + "fake.fake_device(1)\n" + 2 * one
                + "fake.fake_device(0)\n" + one)
    assert [x[:1] + x[1:] if x[0] == "status" else x[0] for x in log] == [
        "asked", ["status", 3], "asked", ["status", 3], "asked", "launch", ["status", 0], "launch",
        ["status", 0], "asked", "launch", ["status", 0], "launch", ["status", 0], "launch",
        ["status", 0]]
    assert [x[3] for x in log if x[0] == "launch"] == [want[0], want[0], want[1], want[1], want[0]]
