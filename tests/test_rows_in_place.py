"""Rotated rows written into a tensor that the call reads other rows of (in place on a fused
projection) or into one tensor: the rule (fa_rows.h, compiled on its own) against a count of the
elements, and what the C ABI takes and refuses. No GPU."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import flash_attention_gb300 as fa
from tests.test_draft_abi import ROTATE, at, lib, rope, struct  # noqa: F401


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    so = tmp_path_factory.mktemp("grids") / "grids.so"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "grids_lib.cpp")
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-o", str(so), src], check=True)
    f = ctypes.CDLL(str(so)).grids_meet
    three = ctypes.c_int64 * 3
    f.argtypes = [three] * 4 + [ctypes.c_int64] * 2
    return lambda na, sa, nb, sb, offset, d=64: bool(
        f(three(*na), three(*sa), three(*nb), three(*sb), offset, d))


def elements(n, st, d, start=0):
    out = set()
    for b in range(n[0]):
        for h in range(n[1]):
            for i in range(n[2]):
                x = start + b * st[0] + h * st[1] + i * st[2]
                out.update(range(x // 8, (x + d) // 8))  # strides and offsets are multiples of 8
    return out


def test_views_of_one_tensor(meet):
    B, n, d = 3, 5, 64
    for H, Hk in ((4, 2), (1, 1), (3, 1), (8, 8)):
        W = (H + 2 * Hk) * d
        st = (n * W, d, W)
        q, k = (B, H, n), (B, Hk, n)
        assert not meet(q, st, k, st, H * d) and not meet(k, st, q, st, -H * d)
        assert not meet(k, st, k, st, Hk * d)
        for off in (0, 8, (H - 1) * d, H * d - 8):
            assert meet(q, st, k, st, off) and meet(k, st, q, st, -off)
        # heads before rows, and batches inside rows
        for st, step in (((H + Hk) * n * d, n * d, d), H * n * d), ((d * (H + Hk), d, B * d * (H + Hk)), H * d):
            assert not meet(q, st, k, st, step) and meet(q, st, k, st, step - 8)
        # a step of the row past the last head: row i of k where row i + 1 of q is
        assert meet(q, (n * W, d, W), k, (n * W, d, W), W)


def test_any_strides(meet):
    r = random.Random(5)
    met = apart = 0
    for _ in range(6000):
        na = [r.randint(1, 4) for _ in range(3)]
        nb = [na[0], r.randint(1, 4), na[2]]
        sa = [8 * r.choice((r.randint(0, 12), r.randint(0, 200))) for _ in range(3)]
        sb = list(sa) if r.random() < 0.6 else [8 * r.randint(0, 120) for _ in range(3)]
        off = 8 * r.randint(-150, 150)
        want = bool(elements(na, sa, 64) & elements(nb, sb, 64, off))
        met, apart = met + want, apart + (not want)
        assert meet(na, sa, nb, sb, off) == want, (na, sa, nb, sb, off)
    assert met > 500 and apart > 500


def test_sizes_of_any_order(meet):
    """Large tensors take no longer, and an answer that would take too many steps is yes."""
    big = (1 << 20, 64, 1 << 10)
    W = 96 * 128
    st = (W << 10, 128, W)
    assert not meet(big, st, (1 << 20, 16, 1 << 10), st, 64 * 128, 128)
    assert meet(big, st, (1 << 20, 16, 1 << 10), st, 63 * 128, 128)
    assert not meet(big, st, big, st, (W << 30) + 128, 128)
    assert meet(big, (8, 16, 24), big, (24, 8, 16), 8, 128)
    assert meet((1, 1, 1), (1 << 50, 1 << 50, 1 << 50), (1, 1, 1), (0, 0, 0), 0)
    assert not meet((1, 1, 1), (1 << 50, 1 << 50, 1 << 50), (1, 1, 1), (0, 0, 0), 64)


FUSED = dict(batch=2, n_heads=32, n_kv_heads=8, rows=4096, head_dim=128)
WIDE = 48 * 128
VIEW = (4096 * WIDE, 128, WIDE)


def fused(lib, back=0, **kw):
    q, k, v = at(0), at(0) + 2 * 32 * 128, at(0) + 2 * 40 * 128
    strides = {n: VIEW for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")}
    d = dict(FUSED, q=q, k=k, q_out=q, k_out=k, **strides)
    d.update(kw)
    return lib.fa_rotary_apply(struct(fa.FaRotaryRows, ROTATE, **d), rope(), back, None)


def no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")


def test_fused_projections_are_taken(lib):
    """Without a GPU the next thing that fails is the device."""
    no_gpu()
    good = [dict(), dict(cu_seqlens=at(30)), dict(batch=1), dict(rows=1),
            # from tensors of their own into one, and out of one
            dict(q=at(20), k=at(25), q_stride=(4096 * 4096, 4096 * 128, 128),
                 k_stride=(4096 * 1024, 4096 * 128, 128)),
            dict(q_out=at(20), k_out=at(25), q_out_stride=(4096 * 4096, 4096 * 128, 128),
                 k_out_stride=(4096 * 1024, 4096 * 128, 128)),
            # heads first in memory
            dict(rows=64, q_stride=(48 * 8192, 8192, 128), k_stride=(48 * 8192, 8192, 128),
                 q_out_stride=(48 * 8192, 8192, 128), k_out_stride=(48 * 8192, 8192, 128),
                 k=at(0) + 2 * 32 * 8192, k_out=at(0) + 2 * 32 * 8192),
            dict(k=None, k_out=None, n_kv_heads=0), dict(k_out=at(0) + 2 * 40 * 128)]
    for kw in good:
        for back in (0, 1):
            assert fused(lib, back, **kw) not in (fa.FA_OK, fa.FA_ERR_INVALID), kw


@pytest.mark.parametrize("kw", [
    dict(q_out=at(0) + 256), dict(q_out=at(0) + 16), dict(k_out=at(0) + 2 * 31 * 128),
    dict(k_out=at(0) + 2 * 33 * 128), dict(q_out=at(0) + 2 * WIDE),
    dict(k_out=at(0) + 2 * 32 * 128 + 2 * WIDE), dict(k_out=at(0) + 2 * (41 * 128 - 8)),
    dict(q_out=at(0) + 2 * 32 * 128, k_out=at(0)),  # one another's places
    dict(n_heads=33), dict(q_out_stride=(4096 * WIDE, 128, WIDE + 128)),
    dict(k_out_stride=(4096 * WIDE, 256, WIDE)),
], ids=str)
def test_rows_on_one_another_are_refused(lib, kw):
    assert fused(lib, **kw) == fa.FA_ERR_INVALID
