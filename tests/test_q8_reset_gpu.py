"""The 8-bit cache's attention after a device reset: its scratch pool, kept between calls, and the
kernels' attributes serve the new context as they served the old one."""
import os
import subprocess
import sys

import pytest

from tests.test_q8_cache_gpu import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# No torch: the reset would end its context. Codes 0x38 are 1.0; 17 keys of equal score.
RESET = """
import ctypes
import sys

import flash_attention_gb300 as fa

for name in ("libcudart.so.13", "/usr/local/cuda/lib64/libcudart.so"):
    try:
        rt = ctypes.CDLL(name)
        break
    except OSError:
        pass
else:
    print("no libcudart")
    sys.exit(0)
lib = fa.load_library()
P, H, ps, d, lens = 4, 2, 16, 128, 17


def device(data):
    p = ctypes.c_void_p()
    assert rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(len(data))) == 0
    assert rt.cudaMemcpy(p, data, ctypes.c_size_t(len(data)), 1) == 0
    return p.value


def call(rows):
    codes = [device(bytes([x]) * (P * H * ps * d)) for x in (0, 0x38)]
    ones = device(bytes(ctypes.c_float(1.0)) * (P * H))
    table, lengths = (device(b"".join(bytes(ctypes.c_int32(x)) for x in y))
                      for y in ([3, 1], [lens]))
    q, o, lse = (device(bytes(H * rows * n)) for n in (2 * d, 2 * d, 4))
    c = fa.FaQ8Cache(*codes, ones, ones, P, H, ps, d, ps, 0)
    p = fa.FaPagedParams(1, H, H, rows, d, ps, 2, P, 0.1, 0, 0, 0)
    assert lib.fa_q8_paged_attention(q, ctypes.byref(c), table, lengths, o, lse,
                                     ctypes.byref(p), None) == fa.FA_OK
    assert lib.fa_device_status(1) == fa.FA_OK
    got = (ctypes.c_uint16 * (H * rows * d))()
    assert rt.cudaMemcpy(got, ctypes.c_void_p(o), ctypes.c_size_t(ctypes.sizeof(got)), 2) == 0
    assert set(got) == {0x3F80}, set(got)


for _ in range(3):
    call(1)
    call(40)
    assert rt.cudaDeviceReset() == 0
"""


def test_calls_after_a_device_reset():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", RESET], cwd=root, capture_output=True, text=True,
                       timeout=300)
    if "no libcudart" in r.stdout:
        pytest.skip("no CUDA runtime library")
    assert r.returncode == 0, r.stderr[-2000:]
