"""The 8-bit cache's writer and reader bit for bit where a warp takes several heads in turn (calls
that fill the GPU many times over), the number of kv heads a multiple of four or not, and pages
smaller than a warp's rows at every head dim that has them."""
import numpy as np
import pytest

from tests import q8_plain as plain
from tests.test_q8_cache_gpu import _gpu, bf16, dev_cache, host_codes, ints  # noqa: F401

pytestmark = pytest.mark.gpu

# Several heads a warp from 152 * 16 warps on, a warp being four heads of 2048 / d rows of K or V:
# total / (2048 / d) * 2 * Hk / 4 of them.
LARGE = [
    # name, Hk, d, page, block, lengths before, new rows of each sequence
    ("hk8", 8, 128, 16, 16, [0, 5, 3], [5000, 4900, 1]),
    ("hk5", 5, 128, 16, 16, [0, 7], [16200, 90]),
    ("hk6_d256", 6, 256, 32, 8, [0, 3], [6000, 700]),
    ("hk10_d64_page8", 10, 64, 8, 8, [0, 13], [15500, 1200]),
    ("hk7_page8_token_scales", 7, 128, 8, 1, [3, 0], [5700, 6000]),
    ("hk4_page256", 4, 128, 256, 256, [100, 0], [9900, 10000]),
]
# the same pages with few rows
SMALL = [
    ("page8", 2, 128, 8, 8, [0, 3, 0, 50, 16], [33, 0, 1, 17, 300]),
    ("page8_block2", 2, 128, 8, 2, [5, 0, 0], [1, 70, 129]),
    ("page8_token_scales", 3, 128, 8, 1, [5, 0, 0], [1, 70, 129]),
    ("page16_d64", 2, 64, 16, 16, [5, 0, 0], [1, 70, 129]),
]


@pytest.mark.parametrize("case", LARGE + SMALL, ids=lambda c: c[0])
def test_write_and_read_match_the_definition(case):
    import torch

    import flash_attention_gb300 as fa

    name, Hk, d, ps, block, past, new = case
    if case in LARGE:
        assert sum(new) // (2048 // d) * 2 * Hk // 4 >= 152 * 16
    rng = np.random.default_rng(len(name) * 7 + d)
    B, total = len(past), sum(new)
    lengths = np.array(past) + new
    per = int(-(-lengths.max() // ps))
    table, P = plain.make_table(rng, B, per)
    cache = plain.make_cache(rng, P, Hk, ps, d, block)
    got = dev_cache(*cache)
    cu = np.concatenate([[0], np.cumsum(new)])
    xs = []
    for _ in range(2):
        x = rng.standard_normal((Hk, total, d)) * np.exp(1.5 * rng.standard_normal((Hk, total, 1)))
        x.reshape(-1)[rng.integers(0, x.size, 50)] = rng.choice([np.inf, -np.inf, np.nan], 50)
        xs.append(bf16(x))
    fa.q8_cache_write(xs[0][0], xs[1][0], *got, ints(table), ints(lengths), cu_seqlens=ints(cu))
    assert fa.fa_device_status(True) == fa.FA_OK
    for w in range(2):
        plain.write(cache[w], cache[2 + w], [xs[w][1][:, cu[b]:cu[b + 1]] for b in range(B)],
                    table, lengths, block)
        np.testing.assert_array_equal(host_codes(got[w]), cache[w])
        np.testing.assert_array_equal(got[2 + w].cpu().numpy(), cache[2 + w])
    # all the keys there are now
    cu = np.concatenate([[0], np.cumsum(lengths)])
    out = fa.q8_cache_read(*got, ints(table), ints(cu), int(cu[-1]))
    assert fa.fa_device_status(True) == fa.FA_OK
    for w in range(2):
        val = plain.values(cache[w], cache[2 + w]).astype(np.float32)
        j = [np.arange(n) for n in lengths]
        want = np.concatenate([val[table[b, x // ps], :, x % ps] for b, x in enumerate(j)])
        want = torch.from_numpy(np.ascontiguousarray(want.transpose(1, 0, 2))).bfloat16()
        assert torch.equal(torch.nan_to_num(out[w].cpu().float(), nan=1e9),
                           torch.nan_to_num(want.float(), nan=1e9))
