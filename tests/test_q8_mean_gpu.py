"""An error that all outputs of the 8-bit cache's attention have in common, which a bound on each
element cannot see: the mean of (o - want) / |want| over a large output with values of one sign.

Bound. An element's own error is at most one bf16 rounding and its weights' 9 bits, 2^-8 + 2^-9 of
|want|, without a preference for either side; over 2^17 elements, 2^9 rows of them at least, with
the weight spread over some 2^7 keys, the mean of the first has a standard deviation below
2^-8 / sqrt(2^17) = 1.1e-5, that of the second, alike for the columns of a row but averaged over
its keys, below 2^-9 / sqrt(2^9 * 2^7) = 0.8e-5. The bound is six times what they make together.
The sequences of a case share their pages.
"""
import numpy as np
import pytest

import oracle
from tests import q8_plain as plain
from tests.test_q8_cache_gpu import A, _gpu, attend, bf16, dev_cache, make_attend  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [
    A("rows2", 32, 32, 16, 1, 128, 16, 16, [2000] * 32),
    A("rows4", 32, 32, 8, 1, 128, 16, 16, [2000] * 32),
    A("rows8_d64", 32, 64, 8, 1, 64, 16, 16, [2000] * 32),
    A("rows16_d256", 32, 4, 1, 4, 256, 16, 16, [2000] * 32),
    A("rows32", 16, 16, 2, 4, 128, 16, 16, [2000] * 16),
    A("rows128", 8, 4, 1, 32, 128, 16, 16, [2000] * 8),
    A("rows128_d64", 16, 4, 1, 32, 64, 16, 16, [2000] * 16),
], ids=lambda c: c["name"])
def test_no_error_in_common(c):
    import flash_attention_gb300 as fa

    rng, table, P, cache, _ = make_attend(dict(c, B=1, lengths=[2000]))
    table = np.repeat(table, c["B"], 0)
    cache[1] &= 0x7F  # values of one sign
    cache[2] /= 4  # scores of a spread of about 1: the weight is that of many keys
    qt, q = bf16(rng.standard_normal((c["B"], c["H"], c["lq"], c["d"])))
    o, _ = attend(c, table, dev_cache(*cache), qt)
    assert fa.fa_device_status(True) == fa.FA_OK
    k, v = (plain.values(cache[w], cache[2 + w]) for w in range(2))
    want, _ = oracle.paged_fwd(q, k, v, table, np.array(c["lengths"]), scale=c["d"] ** -0.5,
                               causal=True)
    assert want.size >= 1 << 17 and want.size // c["d"] >= 1 << 9
    mean = np.mean((o.double().cpu().numpy() - want) / want)
    print(c["name"], mean)
    assert abs(mean) < 8e-5, mean
