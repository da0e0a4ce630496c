"""A launch that fails is reported by the call that made it, and nothing is launched after it.

A process of its own loads tests/launch_stub.cpp in place of the runtime's launches before the library, so no device is
reached: operands are addresses that nothing reads.
"""
import json
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(os.path.dirname(HERE), "spmm_csr_spmv_amd", "libspmm_csr_spmv.so")

RUN = r"""
import ctypes, json, sys
stub = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
L = ctypes.CDLL(sys.argv[2])
p, i32, i64, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
P, BIG, NONE = p(1 << 20), ctypes.c_size_t(1 << 50), p(None)
def norm(rows, H, dt):
    return L.rms_norm(i64(rows), i64(H), i32(dt), P, i64(H), P, i64(H), P, i32(dt), f(1e-6), P, i64(H), P, i64(H), NONE)
def norm_i8(rows, H, dt):
    return L.rms_norm_i8(i64(rows), i64(H), i32(dt), P, i64(H), P, i64(H), P, i32(dt), f(1e-6), P, i64(H), P, i64(H), P, NONE)
def norm_backward(rows, H, dt, dw):
    return L.rms_norm_backward(i64(rows), i64(H), i32(dt), P, i64(H), P, i64(H), P, i32(dt), f(1e-6), P, i64(H), P, i64(H),
                               P if dw else NONE, P, BIG, NONE)
def gemm(S, E, N, K, gate):
    a = [i64(S), i32(E), i64(N), i64(K), i32(1), P, i64(S), i64(K), P if E > 1 else NONE, i32(1), P, i64(K), i64((1 + gate) * N * K),
         P if E > 1 else NONE]
    return L.moe_gated(*a, i32(0), P, i64(2 * N), P, i64(N), NONE) if gate else L.moe_gemm(*a, P, i64(N), NONE)
def backward(S, E, N, K, gate, dA, dB):
    rows = (1 + gate) * N
    a = [P, i64(S), i64(K), P if E > 1 else NONE, i32(1), P, i64(K), i64(rows * K), P if E > 1 else NONE, P if dA else NONE, i64(K),
         P if dB else NONE, i64(K), i64(rows * K), P, BIG, NONE]
    head = [i64(S), i32(E), i64(N), i64(K), i32(1)]
    return (L.moe_gated_backward(*head, i32(0), P, i64(N), P, i64(2 * N), *a) if gate else L.moe_gemm_backward(*head, P, i64(N), *a))
out = []
for name, args in json.loads(sys.argv[3]):
    stub.stub_reset(0)
    rc, n = globals()[name](*args), stub.stub_launches()
    tries = []
    for k in range(1, n + 1):
        stub.stub_reset(k)
        tries.append([globals()[name](*args), stub.stub_launches()])
    out.append([rc, n, tries])
print(json.dumps(out))
"""

# and how many launches each has at least
CALLS = [("norm", (5, 64, 1), 1), ("norm_i8", (5, 9000, 0), 1), ("norm_backward", (700, 64, 1, 1), 2),
         ("norm_backward", (700, 9000, 0, 1), 3), ("norm_backward", (700, 20000, 1, 1), 3), ("norm_backward", (700, 20000, 1, 0), 1),
         ("gemm", (40, 1, 64, 64, 0), 1), ("gemm", (40, 4, 64, 64, 1), 1), ("backward", (16, 1, 4096, 1024, 0, 1, 0), 2),
         ("backward", (32768, 1, 256, 256, 0, 1, 1), 3), ("backward", (2600, 1, 136, 2600, 0, 1, 1), 2),
         ("backward", (9000, 1, 136, 136, 1, 1, 1), 4), ("backward", (4096, 8, 520, 264, 1, 1, 1), 3)]


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(LIB), reason="needs g++ and the built library")
def test_a_failed_launch_is_reported(tmp_path):
    stub = str(tmp_path / "launch_stub.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", os.path.join(HERE, "launch_stub.cpp"), "-o", stub], check=True)
    calls = json.dumps([c[:2] for c in CALLS])
    r = subprocess.run([sys.executable, "-c", RUN, stub, LIB, calls], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    for (name, args, least), (rc, n, tries) in zip(CALLS, json.loads(r.stdout)):
        assert rc == 0 and n >= least, (name, args, rc, n)
        for k, (code, launched) in enumerate(tries, 1):
            assert code == 6 and launched == k, "%s%r: launch %d of %d failed, status %d after %d launches" % (
                name, args, k, n, code, launched)
