"""Per-device set-up against a fake CUDA runtime on the CPU: the W4A4 entry
points set up their own kernels only, and a failure in the set-up of the FP8
linear layer or the cross attention is theirs alone."""
import os
import shutil
import subprocess
import sys

import pytest

from bit_diffusion_transformer_nvfp4_b200 import build

FAKE = r"""
#include <stddef.h>
typedef int err;
int fake_fail, fake_attributes, fake_occupancy, fake_launches;
static int word;
static int encode(void) { return 0; }
err cudaGetDevice(int* d) { *d = 0; return 0; }
err cudaDeviceGetAttribute(int* v, int attr, int d) { (void)d; *v = attr == 75 ? 10 : 148; return 0; }
err cudaGetSymbolAddress(void** p, const void* s) { (void)s; *p = &word; return 0; }
err cudaGetDriverEntryPoint(const char* n, void** f, unsigned long long l, int* q) {
  (void)n; (void)l; *f = (void*)encode; *q = 0; return 0;
}
err cudaFuncSetAttribute(const void* f, int a, int v) { (void)f; (void)a; (void)v; ++fake_attributes; return fake_fail; }
err cudaOccupancyMaxActiveClusters(int* n, const void* f, const void* c) {
  (void)f; (void)c; ++fake_occupancy; *n = 9; return fake_fail;
}
err cudaLaunchKernelExC(const void* c, const void* f, void** a) { (void)c; (void)f; (void)a; ++fake_launches; return 0; }
err cudaGetLastError(void) { return 0; }
"""

PROGRAM = r"""
import ctypes, sys
from ctypes import c_float, c_int64 as i64
fake, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
count = lambda n: ctypes.c_int.in_dll(fake, "fake_" + n)
P = ctypes.c_void_p(1 << 20)
def gemm():
    return lib.w4a4_gemm(P, P, P, None, i64(256), i64(256), i64(256), P, P, P, None, 0, None, 0, P, i64(256), None)
def fp8():
    return lib.fp8_gemm(P, i64(256), P, 1, i64(256), i64(256), i64(256), P, i64(256), P, None, 0, None, i64(0), P, i64(256),
                        None)
def cross():
    return lib.cross_attention_bf16(P, i64(64), P, i64(64), P, i64(64), i64(1), i64(1), i64(9), i64(9), i64(1), i64(1),
                                    i64(64), None, None, i64(0), c_float(0.1), P, i64(64), None)
assert gemm() == 0 and count("launches").value == 1
own = count("attributes").value
assert count("occupancy").value == 0, "a W4A4 call waits for the cross attention's set-up"
if sys.argv[3] == "fails":
    count("fail").value = 1
    assert fp8() == -6 and cross() == -6 and fp8() == -6 and cross() == -6
    count("fail").value = 0
    assert gemm() == 0 and fp8() == -6
else:
    assert fp8() == 0 and count("attributes").value == own + 7
    assert cross() == 0 and count("attributes").value == own + 11 and count("occupancy").value == 8
    assert gemm() == 0 and fp8() == 0 and cross() == 0
    assert count("attributes").value == own + 11 and count("occupancy").value == 8  # once
print("ok")
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
@pytest.mark.parametrize("how", ["works", "fails"])
def test_set_up_of_one_operator_is_not_the_others(tmp_path, how):
    lib = build.build()
    src, fake = tmp_path / "fake.c", tmp_path / "libfake.so"
    src.write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(fake), str(src)], check=True)
    run = subprocess.run([sys.executable, "-c", PROGRAM, str(fake), lib, how], capture_output=True, text=True, timeout=120,
                         env={**os.environ, "LD_PRELOAD": str(fake)})
    assert run.returncode == 0 and run.stdout == "ok\n", run.stdout + run.stderr


def test_in_place_with_another_stride_is_refused():
    """A residual sum or an output over its own input needs the input's rows:
    another stride would overwrite rows before they are read."""
    import ctypes
    from ctypes import c_float, c_int64 as i64
    so = ctypes.CDLL(build.build())
    P, Q = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
    ARG = -8

    def norm(x, r, hidden, ldx, ldr, ldh, rows=4):
        return so.rmsnorm_fp8(x, i64(rows), i64(64), i64(ldx), r, i64(ldr), None, c_float(1e-6), hidden, i64(ldh), None,
                              i64(0), ctypes.c_void_p(1 << 22), i64(64), ctypes.c_void_p(1 << 23), None)

    def linear(r, y, ldr, ldy, rows=4):
        return so.fp8_gemm(P, i64(64), P, 1, i64(rows), i64(64), i64(64), P, i64(64), P, None, 0, r, i64(ldr), y,
                           i64(ldy), None)

    assert norm(P, Q, P, 72, 64, 64) == ARG and norm(Q, P, P, 64, 72, 64) == ARG
    assert norm(P, None, P, 72, 0, 64) == ARG
    assert linear(Q, Q, 72, 64) == ARG and linear(Q, Q, 64, 72) == ARG
    # allowed: the same rows, other memory, one row (asked only where no kernel
    # can start: the addresses are made up)
    if not __import__("torch").cuda.is_available():
        for st in (norm(P, Q, P, 72, 64, 72), norm(Q, P, P, 64, 72, 72), norm(P, Q, None, 72, 64, 0),
                   norm(P, Q, P, 72, 64, 64, rows=1), linear(Q, Q, 72, 72), linear(P, Q, 72, 64),
                   linear(Q, Q, 72, 64, rows=1)):
            assert st == -4
