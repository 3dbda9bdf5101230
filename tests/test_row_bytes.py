"""Four bytes of a row at any address (csrc/row_bytes.cuh, the 8-bit product's loads where K is odd):
the row's bytes, and no byte outside the matrix is touched."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(HERE, "_build", "librowbytes.so")


@pytest.fixture(scope="module")
def probe():
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    subprocess.run(["/usr/local/cuda/bin/nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17",
                    "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(HERE, "..", "block_quantized_expert_gb300", "csrc"),
                    "-o", LIB, os.path.join(HERE, "csrc", "row_bytes_probe.cu")], check=True)
    f = C.CDLL(LIB).probe_row_bytes
    f.argtypes, f.restype = [C.c_void_p] + 6 * [C.c_int] + [C.c_void_p], C.c_uint32
    return f


@pytest.mark.parametrize("start", range(16, 20))
@pytest.mark.parametrize("pad", [0, 1, 6])
def test_inside_the_matrix(probe, start, pad):
    base = np.zeros(300, np.uint8)
    at = -base.ctypes.data % 16  # a 16-byte boundary
    buf = base[at:at + 256]
    buf[:] = np.random.default_rng(start).integers(0, 256, 256)
    for K in (*range(1, 14), 30, 31, 33, 63):
        hi = start + 2 * (K + pad) + K  # three rows
        for r in range(3):
            first = start + r * (K + pad)
            row = buf[first:first + K].astype(np.uint64)
            for c in range(K):
                # `inside` as the kernel has it: words of a row's inner columns
                for inside in (0, 1) if c >= 4 and c + 8 <= K else (0,):
                    marks = np.zeros(256, np.uint8)
                    got = probe(buf.ctypes.data, first, c, K, inside, start, hi, marks.ctypes.data)
                    assert got == sum(int(b) << (8 * i) for i, b in enumerate(row[c:c + 4])), (K, r, c)
                    assert not marks[:start].any() and not marks[hi:].any(), (K, r, c)
                    assert marks[first + c:first + min(c + 4, K)].all()
