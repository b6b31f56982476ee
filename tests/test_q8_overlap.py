"""The 8-bit cache's reader refuses output rows that lie on one another (they would race) and takes
every layout whose rows do not: the rule (fa_rows.h, compiled on its own) against a count of the
elements, and the refusals through the C ABI. No GPU."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import flash_attention_gb300 as fa
from tests.test_q8_abi import FAKE, cache, lib, rows  # noqa: F401

FAR = 1 << 40


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    so = tmp_path_factory.mktemp("rows") / "rows.so"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "rows_lib.cpp")
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-o", str(so), src], check=True)
    f = ctypes.CDLL(str(so)).rows_are_apart
    f.argtypes = [ctypes.c_int64] * 8
    return lambda Hk, total, d, k, v, offset=FAR: bool(f(Hk, total, d, *k, *v, offset))


def elements(Hk, total, d, strides, at=0):
    """The elements of the rows, or None where two rows share one."""
    starts = [at + h * strides[0] + i * strides[1] for h in range(Hk) for i in range(total)]
    seen = set()
    for s in starts:
        seen.update(range(s, s + d))
    return seen if len(seen) == len(starts) * d else None


LAYOUTS = [
    # Hk, total, d, (head stride, row stride), taken
    (2, 8, 128, (256, 128), False),     # head 1's row 0 is head 0's row 2
    (4, 5, 64, (64, 64), False),
    (4, 5, 64, (64, 256), True),        # [total, Hk, d]
    (4, 5, 64, (320, 64), True),        # [Hk, total, d]
    (4, 5, 64, (312, 64), False),       # a head's last row reaches into the next one's first
    (4, 5, 64, (64, 248), False),
    (4, 5, 64, (328, 64), True),
    (2, 9, 64, (64, 128), True),
    (3, 9, 64, (64, 128), False),
    (2, 3, 64, (192, 128), True),       # rows of one head between those of the other
    (3, 4, 64, (192, 128), False),      # two heads on are three rows on
    (1, 5, 64, (0, 64), True),
    (1, 5, 64, (0, 0), False),
    (5, 1, 64, (64, 0), True),
    (5, 1, 64, (0, 64), False),
    (1, 1, 64, (0, 0), True),
]


@pytest.mark.parametrize("case", LAYOUTS, ids=str)
def test_rows_on_one_another(lib, rule, case):
    Hk, total, d, st, taken = case
    assert (elements(Hk, total, d, st) is not None) == taken
    good = (d * total, d)
    for k, v in ((st, good), (good, st)):
        assert rule(Hk, total, d, k, v) == taken
        if not taken:
            r = rows(lengths=None, total=total, k_stride=(0, *k), v_stride=(0, *v), v=FAKE + FAR)
            assert lib.fa_q8_cache_read(cache(n_kv_heads=Hk, head_dim=d), r, None) == \
                fa.FA_ERR_INVALID


def test_any_strides(rule):
    r = random.Random(1)
    taken = 0
    for _ in range(3000):
        Hk, total, d = r.randint(1, 6), r.randint(1, 9), 64
        st = (8 * r.randint(0, 60), 8 * r.randint(0, 60))
        want = elements(Hk, total, d, st) is not None
        taken += want
        assert rule(Hk, total, d, st, (d * total, d)) == want, (Hk, total, st)
    assert 100 < taken < 2900


def test_keys_and_values_on_one_another(lib, rule):
    """K and V of the same strides: the halves of one tensor are taken, in either order; the same
    rows, and rows that reach into the other's, are not."""
    Hk, total, d = 3, 7, 64

    def refused(k, v, k_at, v_at, Hk=Hk, total=total):
        assert not rule(Hk, total, d, k, v, (v_at - k_at) // 2)
        rr = rows(lengths=None, total=total, k_stride=(0, *k), v_stride=(0, *v), k=k_at, v=v_at)
        assert lib.fa_q8_cache_read(cache(n_kv_heads=Hk, head_dim=d), rr, None) == \
            fa.FA_ERR_INVALID

    for st, half in (((2 * d * total, d), d * total), ((d, 2 * d * Hk), d * Hk),
                     ((2 * d, 2 * d * Hk), d), ((d, d * Hk), d * Hk * total)):
        assert rule(Hk, total, d, st, st, half) and rule(Hk, total, d, st, st, -half)
        for near in (0, 8, half - 8):
            assert elements(Hk, total, d, st) & elements(Hk, total, d, st, near)
            refused(st, st, FAKE, FAKE + 2 * near)
            refused(st, st, FAKE + 2 * near, FAKE)
    # strides of dimensions of one row or head do not count
    refused((0, d), (999 * 8, d), FAKE, FAKE, Hk=1)
    refused((d, 0), (d, 999 * 8), FAKE, FAKE, total=1)
    # of different strides: at one address
    refused((d * total, d), (d, d * Hk), FAKE, FAKE)


def test_any_offset_of_keys_and_values(rule):
    r = random.Random(2)
    taken = refused = 0
    while taken < 300 or refused < 300:
        Hk, total, d = r.randint(1, 5), r.randint(1, 7), 64
        st = (8 * r.randint(8, 80), 8 * r.randint(8, 80))
        k = elements(Hk, total, d, st)
        if k is None:
            continue
        off = 8 * r.randint(-100, 100)
        want = not (k & elements(Hk, total, d, st, off))
        taken, refused = taken + want, refused + (not want)
        assert rule(Hk, total, d, st, st, off) == want, (Hk, total, st, off)


def test_no_rows_and_strides_of_any_size(rule):
    assert rule(2, 0, 64, (64, 64), (64, 64), 0)
    assert not rule(2, 3, 64, (1 << 62, 64), (1 << 62, 64))
    assert rule(1, 3, 64, (1 << 62, 64), (1 << 62, 64))
    assert rule(1 << 20, 1 << 20, 64, (64 << 20, 64), (64 << 20, 64), 1 << 48)
