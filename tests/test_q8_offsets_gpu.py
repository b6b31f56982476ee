"""The 8-bit cache's writer and reader with packed offsets out of range: they are reported wherever
in the batch they are, nothing is written but the pages of the batch and the rows of the outputs,
and sequences whose offsets are in order come out as they would alone."""
import numpy as np
import pytest

from tests import q8_plain as plain
from tests.test_q8_cache_gpu import _gpu, bf16, dev_cache, host_codes, ints  # noqa: F401

pytestmark = pytest.mark.gpu

# offsets, rows there are, and the sequences that come out right: all of them where the offsets do
# not decrease (clamped to the rows there are)
OFFSETS = [
    ("past_the_end", [0, 5, 9, 15, 40], 20, [0, 1, 2]),
    ("below_zero", [-3, 5, 9, 15, 20], 20, [1, 2, 3]),
    ("decreasing", [0, 9, 5, 15, 20], 20, []),
    ("decreasing_by_far", [0, 90, 20, 100], 100, []),
    # one entry among many, between those that a search by halves or by 32nds looks at
    ("hidden", [0, 1000] + [0] * 62 + [1000], 1000, []),
    ("hidden_late", [0] * 61 + [900, 0, 1000], 1000, []),
    ("hidden_of_1500", [0] * 1001 + [900] + [0] * 498 + [1000], 1000, []),
]


@pytest.mark.parametrize("case", OFFSETS, ids=lambda c: c[0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_write_with_offsets_out_of_range(case, d):
    import flash_attention_gb300 as fa

    name, cu, total, fine = case
    rng = np.random.default_rng(len(name) + d)
    B, Hk, ps, block = len(cu) - 1, 2, 16, 16
    clamped = np.clip(cu, 0, total)
    lengths = np.maximum(np.diff(clamped), 0) + 3
    per = -(-int(lengths.max()) // ps) if B < 10 else 1
    if B >= 10:
        lengths[:] = 16
    table, P = plain.make_table(rng, B, per, spare=9)
    cache = plain.make_cache(rng, P, Hk, ps, d, block)
    got = dev_cache(*cache)
    x = [bf16(rng.standard_normal((Hk, total, d))) for _ in range(2)]
    fa.q8_cache_write(x[0][0], x[1][0], *got, ints(table), ints(lengths), cu_seqlens=ints(cu))
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    others = np.setdiff1d(np.arange(P), table)
    for w in range(2):
        codes, scales = host_codes(got[w]), got[2 + w].cpu().numpy()
        np.testing.assert_array_equal(codes[others], cache[w][others])
        np.testing.assert_array_equal(scales[others], cache[2 + w][others])
        plain.write(cache[w], cache[2 + w],
                    [x[w][1][:, max(a, 0):max(b, a, 0)] for a, b in zip(clamped, clamped[1:])],
                    table, lengths, block)
        for b in fine:
            np.testing.assert_array_equal(codes[table[b]], cache[w][table[b]])
            np.testing.assert_array_equal(scales[table[b]], cache[2 + w][table[b]])


@pytest.mark.parametrize("case", OFFSETS, ids=lambda c: c[0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_read_with_offsets_out_of_range(case, d):
    import torch

    import flash_attention_gb300 as fa

    name, cu, total, fine = case
    rng = np.random.default_rng(len(name) + d)
    B, Hk, ps, pad = len(cu) - 1, 2, 16, 16
    clamped = np.clip(cu, 0, total)
    per = -(-total // ps)
    table, P = plain.make_table(rng, B, per) if B < 10 else \
        (rng.integers(0, 100, (B, per)).astype(np.int32), 100)
    cache = plain.make_cache(rng, P, Hk, ps, d, 16)
    # the outputs are the middle of filled buffers
    whole = [torch.full((Hk, total + 2 * pad, d), 7.0, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    out = tuple(t[:, pad:pad + total] for t in whole)
    fa.q8_cache_read(*dev_cache(*cache), ints(table), ints(cu), total, out=out)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    for w in range(2):
        assert (whole[w][:, :pad] == 7).all() and (whole[w][:, pad + total:] == 7).all()
        val = plain.values(cache[w], cache[2 + w]).astype(np.float32)
        for b in fine:
            j = np.arange(clamped[b + 1] - clamped[b])
            want = torch.from_numpy(val[table[b, j // ps], :, j % ps].transpose(1, 0, 2))
            assert torch.equal(out[w][:, clamped[b]:clamped[b + 1]].cpu(), want.bfloat16())


def test_offsets_in_order_are_not_reported():
    import torch

    import flash_attention_gb300 as fa

    for B in (1, 33, 1500):
        cu = np.linspace(0, 700, B + 1).astype(int)
        lengths = np.maximum(np.diff(cu), 1)
        per = -(-int(lengths.max()) // 16)
        cache = fa.make_q8_cache(B * per, 2, 16, 64)
        table = ints(np.arange(B * per).reshape(B, per))
        x = torch.randn(2, 700, 64, device="cuda").bfloat16()
        fa.q8_cache_write(x, x, *cache, table, ints(lengths), cu_seqlens=ints(cu))
        fa.q8_cache_read(*cache, table, ints(cu), 700)
        assert fa.fa_device_status(True) == fa.FA_OK
