"""The stretched frequencies pair by pair. No GPU."""
import math

import pytest

import flash_attention_gb300 as fa

torch = pytest.importorskip("torch")


def turns_to_pair(n, base, length, turns):
    """i with base^(2 i / n) * 2 pi * turns = length, by bisection."""
    lo, hi = -50.0 * n, 50.0 * n
    for _ in range(200):
        mid = (lo + hi) / 2
        if 2 * mid / n * math.log(base) + math.log(2 * math.pi * turns) < math.log(length):
            lo = mid
        else:
            hi = mid
    return lo


@pytest.mark.parametrize("n,base,factor,length,fast,slow", [
    (128, 10000.0, 4.0, 4096, 32.0, 1.0), (64, 500000.0, 8.0, 8192, 32.0, 1.0),
    (96, 10000.0, 2.5, 2048, 16.0, 2.0), (128, 10000.0, 16.0, 1 << 20, 32.0, 1.0),
    (64, 10000.0, 4.0, 40, 32.0, 1.0), (16, 10.0, 3.0, 100, 1.01, 1.0)])
def test_parts(n, base, factor, length, fast, slow):
    """Frequency i is f_i (1 - r) + f_i / factor r with r rising linearly from the whole i at or below
    which `fast` turns are made to the one at or above which `slow` are, within 0 .. n - 1; a step where
    the two are one."""
    got, scale = fa.rotary_inv_freq(n, base, factor=factor, method="parts", original_len=length,
                                    beta_fast=fast, beta_slow=slow, device="cpu")
    low = max(math.floor(turns_to_pair(n, base, length, fast) + 1e-9), 0)
    high = min(math.ceil(turns_to_pair(n, base, length, slow) - 1e-9), n - 1)
    for i, f in enumerate(got.tolist()):
        r = float(i > low) if high == low else min(max((i - low) / (high - low), 0.0), 1.0)
        want = base ** (-2 * i / n) * ((1 - r) + r / factor)
        assert abs(f / want - 1) < 1e-12, (i, r)
    assert scale == 0.1 * math.log(factor) + 1


def test_base():
    """The base that makes the slowest pair factor times as slow."""
    n, base, factor = 128, 10000.0, 8.0
    got, scale = fa.rotary_inv_freq(n, base, factor=factor, method="base", device="cpu")
    new = (base ** ((n - 2) / n) * factor) ** (n / (n - 2))
    for i, f in enumerate(got.tolist()):
        assert abs(f * new ** (2 * i / n) - 1) < 1e-12
    assert scale == 1.0
