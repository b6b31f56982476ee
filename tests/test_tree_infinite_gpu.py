"""Tree attention where values of keys before the tree are not finite: every row that sees such a key
has the value added as it is, whatever its weight, in every variant, in whole units and in cut ones.
The comparison and its tolerance are tests.test_tree_gpu.check's (not finite elements: equal)."""
import numpy as np
import pytest

from tests import draft_plain as plain
from tests.test_rotary_gpu import _gpu, bf16, ints  # noqa: F401
from tests.test_tree_gpu import check, make, masks

pytestmark = pytest.mark.gpu

ROWS = [  # d, query heads of a kv head, nodes
    (64, 1, 8), (64, 4, 8), (64, 3, 11), (64, 4, 16), (64, 5, 13), (64, 4, 32), (64, 5, 26),
    (128, 1, 8), (128, 4, 32), (128, 5, 26), (256, 1, 8), (256, 5, 26),
]
LENGTHS = {"whole": [400, 70, 40], "cut": [3000, 700, 40]}


def run(d, G, T, lengths, far, bad_page=False):
    """far: half of the keys have scores 160 below the others' (weights of 2^-230: 0 in 32 bits, and
    not in 64), among them whole tiles, a half of each tile, and whole shares of cut units."""
    import torch

    import flash_attention_gb300 as fa

    B, Hk, ps, scale = len(lengths), 2, 16, 0.125
    rng, table, (_, kx), (_, vx), (_, qx) = make(d + T, B, G * Hk, Hk, T, d, ps, lengths)
    m = masks(rng, B, T, "trees")
    qx[..., 0] = 8
    P = kx.shape[0]
    for b, n in enumerate(lengths):
        j = np.arange(n)
        low = (j < 128) | (j < n // 2) | (j % 64 < 32) if far else j < 0
        low &= j < n - T - 1
        kx[table[b][j // ps], :, j % ps, 0] = np.where(low, -160.0, 0.0)[:, None]
        before = n - T  # keys before the tree
        normal = np.flatnonzero(~low[:before])

        def put(key, column, value):
            vx[table[b][key // ps], :, key % ps, column] = value

        put(0, 1, np.inf)
        put(normal[0], 2, np.inf)
        put(normal[-1], 3, -np.inf)
        put(0, 4, np.inf)
        put(before - 1, 4, -np.inf)
        put(before // 2, 5, np.nan)
        for key in (0, before // 3, before // 2, before - 1):
            put(key, 20, -np.inf)
        put(1, d - 1, np.inf)  # and a node that some rows see, with the other sign
        put(n - T // 2, d - 1, -np.inf)
        put(n - 1, d - 2, np.inf)
    (kc, kx), (vc, vx), (q, qx) = bf16(kx), bf16(vx), bf16(qx)
    if bad_page:
        table[0, 3] = P
        table[1, 1] = -1
    want = plain.tree_attention(qx, kx, vx, table, lengths, m, scale)
    for kind in (np.isposinf, np.isneginf, np.isnan):
        assert kind(want[0]).any()
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda(),
                                  scale=scale)
    assert fa.fa_device_status(True) == (fa.FA_ERR_BAD_INPUT if bad_page else fa.FA_OK)
    check(got, want)


@pytest.mark.parametrize("far", [False, True], ids=["near", "far"])
@pytest.mark.parametrize("units", ["whole", "cut"])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_values_before_the_tree_are_added_as_they_are(case, units, far):
    run(*case, LENGTHS[units], far)


@pytest.mark.parametrize("units", ["whole", "cut"])
@pytest.mark.parametrize("d", [64, 128])
def test_beside_pages_outside_the_cache(d, units):
    """Keys of such pages are zeros, and nothing is read there."""
    run(d, 2, 8, LENGTHS[units], False, True)


@pytest.mark.parametrize("d,T", [(64, 8), (64, 20), (128, 8), (256, 8)])
def test_a_value_that_is_nan_everywhere_or_a_query(d, T):
    """All values NaN; a query of NaN takes its own row alone."""
    import torch

    import flash_attention_gb300 as fa

    lengths = [900, 30]
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(d, 2, 4, 2, T, d, 16, lengths)
    m = masks(rng, 2, T, "trees")
    qx[0, 1, 3] = np.nan
    vx[table[1]] = np.nan
    (vc, vx), (q, qx) = bf16(vx), bf16(qx)
    with np.errstate(invalid="ignore"):
        want = plain.tree_attention(qx, kx, vx, table, lengths, m, 0.1)
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda(),
                                  scale=0.1)
    check(got, want)


@pytest.mark.parametrize("units", ["whole", "cut"])
@pytest.mark.parametrize("d,G,T", [(64, 1, 8), (64, 5, 26), (128, 4, 32), (256, 1, 8)])
def test_without_lse(d, G, T, units):
    """The C call that asks for no L gives the same bits, NaN scores and infinite values alike."""
    import ctypes

    import torch

    import flash_attention_gb300 as fa

    lengths, Hk, ps = LENGTHS[units], 2, 16
    B, H = len(lengths), G * Hk
    rng, table, (_, kx), (_, vx), (_, qx) = make(d, B, H, Hk, T, d, ps, lengths)
    qx[0, :, 2] = np.nan
    vx[table[0, 1], :, 3] = np.inf  # all columns of a key
    vx[table[1, 0], :, 5, :7] = -np.inf
    (kc, _), (vc, _), (q, _) = bf16(kx), bf16(vx), bf16(qx)
    m = torch.from_numpy(np.broadcast_to(masks(rng, B, T, "trees"), (B, T, T)).copy()).cuda()
    tb, lens = ints(table), ints(lengths)
    want, lse = fa.paged_tree_attention(q, kc, vc, tb, lens, m, scale=0.1)
    assert want.isinf().any() and want.isnan().any() and lse[0, :, 2].isnan().all()
    assert want[0, :, 2].isnan().all()
    o = torch.full_like(q, 7.0)
    p = fa.FaPagedParams(B, H, Hk, T, d, ps, table.shape[1], kc.shape[0], 0.1, 0, 0, 0)
    rc = fa.load_library().fa_paged_tree_attention(
        q.data_ptr(), kc.data_ptr(), vc.data_ptr(), tb.data_ptr(), lens.data_ptr(), m.data_ptr(),
        T * T, o.data_ptr(), None, ctypes.byref(p), torch.cuda.current_stream().cuda_stream)
    assert rc == fa.FA_OK
    assert torch.equal(o.nan_to_num(9.0), want.nan_to_num(9.0))
    assert torch.equal(o.isnan(), want.isnan()) and torch.equal(o.isinf(), want.isinf())
