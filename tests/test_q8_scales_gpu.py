"""Attention over the 8-bit cache with value scales far apart within one row: a key's share of the
softmax's sum does not depend on its value's scale, and its value counts beside values whose scale
is up to 2^200 times as large.

Tolerances, per element. O: one bf16 rounding (2^-8 of |o|), and of sum_j p_j |v_j| the weights' 9
bits (2^-9) and 2^-13: what the f32 arithmetic adds is four roundings of numbers of up to 2^8 in
base 2 (log2 of the scale less m, the score on top of it, and for the sum that scale and the sum's
unit taken out again), 2^-17 each, in the weights and in the sum, times ln 2, and the 2^-14 of
test_q8_cache_gpu.py. L: the same four and two more where m and the sum are put together, 6 * 2^-17
below 2^-14.
"""
import numpy as np
import pytest

import oracle
from tests import q8_plain as plain
from tests.test_q8_cache_gpu import (A, _gpu, attend, bf16, dev_cache, ints,  # noqa: F401
                                     make_attend)

pytestmark = pytest.mark.gpu

# decode and several new positions in blocks of 8 and 16 rows, chunks in blocks of 128; units cut
# over many CTAs, and (many sequences) mostly whole ones
SHAPES = [
    A("one_row", 2, 2, 2, 1, 128, 16, 1, [3000, 4500]),
    A("one_row_d64", 2, 2, 2, 1, 64, 16, 1, [3000, 4500]),
    A("one_row_d256", 2, 8, 2, 1, 256, 32, 1, [700, 4500]),
    A("rows8_block8", 2, 8, 1, 1, 128, 16, 8, [3000, 4500]),
    A("rows16", 2, 8, 2, 4, 128, 16, 1, [300, 2500]),
    A("whole_units", 200, 2, 2, 1, 128, 16, 1, [150] * 200),
    A("whole_units_rows16", 200, 8, 2, 4, 64, 16, 1, [150] * 200),
    A("chunk", 2, 4, 1, 32, 128, 16, 1, [3000, 1500]),
    A("chunk_d64", 2, 4, 1, 32, 64, 16, 1, [3000, 1500]),
    A("chunk_block8", 2, 4, 1, 32, 128, 16, 8, [3000, 1500]),
    A("chunk_whole_units", 80, 2, 2, 40, 64, 16, 1, [300] * 80),
    A("chunk_whole_units_d128", 80, 2, 2, 40, 128, 16, 1, [300] * 80),
]


def scales_at(kind, rng, n, block):
    """log2 of the value scales of the blocks of n positions."""
    m = -(-n // block)
    j = np.arange(m) / m
    if kind == "rising":
        return np.where(j < 0.5, -100, 60)
    if kind == "falling":
        return np.where(j < 0.5, 60, -100)
    if kind == "steps":  # the maximum moves by 40 each time
        return -100 + 40 * (j * 6).astype(int)
    if kind == "two":  # as a zero block (2^-100) beside values of 10^10
        return np.where(rng.random(m) < 0.5, -100, 30)
    return rng.choice([-100, -60, 0, 40, 100], m)


@pytest.mark.parametrize("kind", ["rising", "falling", "steps", "two", "mixed"])
@pytest.mark.parametrize("c", SHAPES, ids=lambda c: c["name"])
def test_value_scales_far_apart(c, kind):
    import flash_attention_gb300 as fa

    rng, table, P, cache, q = make_attend(c)
    v = plain.VALUES[cache[1]]
    cache[1][:] = plain.to_code(np.where(v < 0, v - 8, v + 8).clip(-448, 448))  # none is zero
    for b, n in enumerate(c["lengths"]):
        e = scales_at(kind, rng, n, c["block"])
        j = np.arange(e.size) * c["block"]
        cache[3][table[b, j // c["ps"]], :, j % c["ps"] // c["block"]] = (2.0 ** e)[:, None]
    qt, q = bf16(q)
    o, lse = attend(c, table, dev_cache(*cache), qt)
    assert fa.fa_device_status(True) == fa.FA_OK
    k, v = (plain.values(cache[w], cache[2 + w]) for w in range(2))
    kw = dict(scale=c["d"] ** -0.5, causal=True)
    want, l_want = oracle.paged_fwd(q, k, v, table, np.array(c["lengths"]), **kw)
    mass, _ = oracle.paged_fwd(q, k, np.abs(v), table, np.array(c["lengths"]), **kw)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -13) * mass
    l_used = np.max(np.abs(lse.double().cpu().numpy() - l_want)) * 2 ** 14
    used = np.max(np.abs(o.double().cpu().numpy() - want) / tol)
    assert used <= 1 and l_used <= 1, (used, l_used)


def test_a_zero_block_before_large_values():
    """What the writer makes of values of zero and of 10^12, at equal scores: O is their mean."""
    import torch

    import flash_attention_gb300 as fa

    d, ps = 128, 16
    for lq in (1, 40):
        for n in (32, 256, 4096):  # in one tile, in two, over many CTAs
            cache = fa.make_q8_cache(n // ps, 1, ps, d)
            table = ints(np.arange(n // ps)[None])
            k = torch.zeros(1, n, d, dtype=torch.bfloat16, device="cuda")
            v = torch.zeros_like(k)
            v[:, n // 2:] = 2.0 ** 40
            fa.q8_cache_write(k, v, *cache, table, ints([n]), cu_seqlens=ints([0, n]))
            q = torch.zeros(1, 1, lq, d, dtype=torch.bfloat16, device="cuda")
            o, lse = fa.q8_paged_attention(q, *cache, table, ints([n]), scale=1.0, causal=False)
            assert fa.fa_device_status(True) == fa.FA_OK
            assert (o == 2.0 ** 39).all(), o.float().flatten()[:4]
            assert (lse - np.log(n)).abs().max() < 2.0 ** -14


# --------------------------------------------------------------------- scales out of range
@pytest.mark.parametrize("lq,d,block", [(1, 128, 16), (1, 128, 1), (1, 64, 8), (3, 256, 2),
                                        (4, 128, 1), (20, 64, 16), (20, 128, 1)])
def test_scales_out_of_range_are_reported(lq, d, block):
    """The attention admits scales in [0, 2^100]: another one is reported where a key that is read
    has it, for keys and for values, and nowhere else."""
    import flash_attention_gb300 as fa

    c = A("range", 2, 4, 2, lq, d, 16, block, [300, 133])
    _, table, P, cache, q = make_attend(c)
    qt, _ = bf16(q)
    nb = 16 // block
    for which in (2, 3):
        for value in (2.0 ** 101, np.inf, np.nan, -1.0):
            for b, pos in ((0, 0), (0, 299), (1, 77)):
                bad = [x.copy() for x in cache]
                bad[which][table[b, pos // 16], 1, pos % 16 // block] = value
                attend(c, table, dev_cache(*bad), qt)
                assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT, (which, value, b, pos)
            bad = [x.copy() for x in cache]  # behind the end: 133 keys end in the 9th page
            first = 133 % 16 // block + 1  # the first block without a key
            bad[which][table[1, 8], :, first:nb] = value
            bad[which][np.setdiff1d(np.arange(P), np.concatenate(
                [table[0, :19], table[1, :9]]))] = value
            attend(c, table, dev_cache(*bad), qt)
            assert fa.fa_device_status(True) == fa.FA_OK, (which, value)
    edge = [x.copy() for x in cache]
    edge[2][:, :, 0], edge[3][:, :, 0] = 0.0, 0.0
    attend(c, table, dev_cache(*edge), qt)
    edge[3][:, :, 0] = 2.0 ** 100
    attend(c, table, dev_cache(*edge), qt)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_values_that_the_attention_does_not_admit():
    """The writer takes any finite value (up to a scale of 2^120); the attention over it says so."""
    import torch

    import flash_attention_gb300 as fa

    for size, status in ((5e32, fa.FA_OK), (6e32, fa.FA_ERR_BAD_INPUT),
                         (3e38, fa.FA_ERR_BAD_INPUT)):
        for which in (0, 1):
            for lq in (1, 40):
                cache = fa.make_q8_cache(2, 1, 16, 64)
                x = [torch.ones(1, 1, 5, 64, dtype=torch.bfloat16, device="cuda")
                     for _ in range(2)]
                x[which][0, 0, 3, 7] = size
                fa.q8_cache_write(*x, *cache, ints([[1]]), ints([5]))
                assert fa.fa_device_status(True) == fa.FA_OK
                q = torch.zeros(1, 1, lq, 64, dtype=torch.bfloat16, device="cuda")
                fa.q8_paged_attention(q, *cache, ints([[1]]), ints([5]), scale=1.0)
                assert fa.fa_device_status(True) == status, (size, which, lq)
