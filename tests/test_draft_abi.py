"""The entry points of a drafted decoding step without a GPU: every bad argument is refused before the
device or any pointer is touched, the binding's own checks, and the plain forms that the GPU tests
compare with, against other ways to the same numbers."""
import ctypes
import math

import numpy as np
import pytest

import flash_attention_gb300 as fa
from tests import draft_plain as plain

FAKE = 0x10000000  # aligned, never dereferenced: checks come first


def at(i):  # tensors that do not meet
    return FAKE * (i + 1)


ROPE = dict(inv_freq=at(20), positions=None, pos_stride=0, rotary_dim=64, interleaved=0, offset=0,
            scale=1.0)
ROTATE = dict(q=at(0), k=at(1), q_out=at(2), k_out=at(3), q_stride=(4096, 1024, 128),
              k_stride=(2048, 1024, 128), q_out_stride=(4096, 1024, 128),
              k_out_stride=(2048, 1024, 128), cu_seqlens=None, batch=2, n_heads=4, n_kv_heads=2,
              rows=8, head_dim=128, reserved=0)
APPEND = dict(k=at(0), v=at(1), q=at(2), q_out=at(3), k_cache=at(4), v_cache=at(5),
              k_stride=(2048, 1024, 128), v_stride=(2048, 1024, 128), q_stride=(4096, 1024, 128),
              cu_seqlens=None, block_table=at(6), lengths=at(7), batch=2, n_heads=4, n_kv_heads=2,
              head_dim=128, page_size=16, max_pages=4, num_pages=10, total=0, new_len=8, reserved=0)
KEPT = dict(k_cache=at(0), v_cache=at(1), block_table=at(2), lengths=at(3), keep=at(4), counts=at(5),
            new_lengths=at(6), batch=2, n_kv_heads=2, head_dim=128, page_size=16, max_pages=4,
            num_pages=10, tree_len=8, max_keep=4)
PARAMS = dict(batch=2, n_heads=8, n_kv_heads=2, q_len=8, head_dim=128, page_size=16, max_pages=4,
              num_pages=10, scale=0.1, causal=0, num_splits=0, reserved=0)

BAD_ROPE = [dict(inv_freq=None), dict(inv_freq=at(20) + 4), dict(positions=FAKE + 2),
            dict(pos_stride=-1, positions=FAKE), dict(pos_stride=8), dict(rotary_dim=0),
            dict(rotary_dim=24), dict(rotary_dim=144), dict(interleaved=2),
            dict(offset=3, positions=FAKE), dict(scale=float("nan")), dict(scale=float("inf"))]
BAD_ROTATE = [
    dict(q=None), dict(q=at(0) + 8), dict(k=None), dict(k_out=None), dict(q_out=at(2) + 2),
    dict(q_stride=(4096, 1024, 127)), dict(k_stride=(-8, 1024, 128)), dict(batch=0),
    dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=-1), dict(rows=-1), dict(head_dim=96),
    dict(reserved=1), dict(batch=1 << 20, rows=1 << 20), dict(cu_seqlens=FAKE + 2),
    dict(n_heads=65535),
    # outputs on inputs, on one another, and rows on rows
    dict(q_out=at(0) + 16), dict(q_out=at(1)), dict(k_out=at(0)), dict(k_out=at(2)),
    dict(q_out=at(0), q_out_stride=(4096, 128, 512)), dict(q_out_stride=(4096, 1024, 64)),
    dict(q_out_stride=(4096, 1016, 128)), dict(q_out_stride=(0, 1024, 128)),
    dict(q_out_stride=(4088, 1024, 128)), dict(k_out_stride=(1 << 60, 1024, 128)),
]
BAD_APPEND = [
    dict(k=None), dict(v=at(1) + 8), dict(q=None), dict(q_out=None), dict(q_out=at(3) + 8),
    dict(k_cache=None), dict(v_cache=at(5) + 8), dict(k_stride=(2048, 1024, 4)),
    dict(v_stride=(2048, -1024, 128)), dict(q_stride=(4096, 1 << 60, 128)),
    dict(block_table=None), dict(block_table=at(6) + 1), dict(lengths=None), dict(lengths=at(7) + 2),
    dict(cu_seqlens=at(8) + 2, total=8, new_len=0), dict(batch=0), dict(n_heads=0), dict(n_heads=-1),
    dict(n_kv_heads=0), dict(head_dim=32), dict(page_size=12), dict(page_size=4),
    dict(page_size=512), dict(max_pages=0), dict(max_pages=1 << 19), dict(num_pages=0),
    dict(num_pages=1 << 30), dict(total=8), dict(new_len=0), dict(new_len=1 << 23),
    dict(cu_seqlens=at(8), total=-1, new_len=0), dict(cu_seqlens=at(8), total=8, new_len=8),
    dict(batch=1 << 20, new_len=1 << 20), dict(reserved=1), dict(n_heads=65534),
    dict(q_out=at(2)), dict(q_out=at(0)), dict(q_out=at(1)), dict(q_out=at(4)), dict(q_out=at(5)),
    dict(k=at(4)), dict(k=at(5)), dict(v=at(4) + 16), dict(v=at(5)), dict(q=at(4)), dict(q=at(5)),
    dict(v_cache=at(4)),
]
BAD_KEPT = [
    dict(k_cache=None), dict(v_cache=at(1) + 8), dict(block_table=None), dict(lengths=at(3) + 1),
    dict(keep=None), dict(keep=at(4) + 2), dict(counts=None), dict(counts=at(5) + 2),
    dict(new_lengths=None), dict(new_lengths=at(6) + 2), dict(batch=0), dict(n_kv_heads=0),
    dict(head_dim=96), dict(page_size=24), dict(max_pages=1 << 19), dict(num_pages=0),
    dict(tree_len=0), dict(tree_len=257), dict(max_keep=0), dict(max_keep=9),
    dict(new_lengths=at(3)), dict(new_lengths=at(3) + 4), dict(new_lengths=at(5)),
    dict(new_lengths=at(4) + 12), dict(new_lengths=at(2)), dict(n_kv_heads=1 << 20, num_pages=1),
]
BAD_PARAMS = [dict(batch=0), dict(n_heads=7), dict(q_len=0), dict(q_len=257), dict(scale=0.0),
              dict(causal=1), dict(num_splits=1), dict(reserved=1), dict(head_dim=96),
              dict(page_size=12), dict(num_pages=0), dict(max_pages=0), dict(max_pages=1 << 19),
              dict(batch=40000)]


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load_library()


def rope(**kw):
    return ctypes.byref(fa.FaRotary(**dict(ROPE, **kw)))


def params(**kw):
    return ctypes.byref(fa.FaPagedParams(**dict(PARAMS, **kw)))


def struct(cls, base, **kw):
    d = dict(base, **kw)
    for n in d:
        if n.endswith("_stride") and n != "pos_stride":
            d[n] = (ctypes.c_int64 * 3)(*d[n])
    return ctypes.byref(cls(**d))


def ids(kw):
    return ",".join(f"{k}={v}" for k, v in kw.items())


@pytest.mark.parametrize("kw", BAD_ROPE, ids=ids)
def test_bad_rotations_are_refused(lib, kw):
    r = rope(**kw)
    assert lib.fa_rotary_apply(struct(fa.FaRotaryRows, ROTATE), r, 0, None) == fa.FA_ERR_INVALID
    assert lib.fa_paged_append(struct(fa.FaPagedRows, APPEND), r, None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", BAD_ROTATE, ids=ids)
def test_bad_rows_are_refused(lib, kw):
    rows = struct(fa.FaRotaryRows, ROTATE, **kw)
    assert lib.fa_rotary_apply(rows, rope(), 0, None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", BAD_APPEND, ids=ids)
def test_bad_appends_are_refused(lib, kw):
    rows = struct(fa.FaPagedRows, APPEND, **kw)
    assert lib.fa_paged_append(rows, rope(), None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", BAD_KEPT, ids=ids)
def test_bad_keeps_are_refused(lib, kw):
    assert lib.fa_paged_keep(struct(fa.FaPagedKept, KEPT, **kw), None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", BAD_PARAMS, ids=ids)
def test_bad_tree_parameters_are_refused(lib, kw):
    p = params(**kw)
    assert lib.fa_paged_tree_attention(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, None, p,
                                       None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("i,value", [(0, None), (1, FAKE + 8), (2, None), (3, FAKE + 2), (4, None),
                                     (5, None), (6, -1), (7, FAKE + 2), (8, FAKE + 1), (9, None)])
def test_bad_tree_arguments_are_refused(lib, i, value):
    args = [FAKE] * 6 + [0, FAKE, None, params(), None]
    args[i] = value
    assert lib.fa_paged_tree_attention(*args) == fa.FA_ERR_INVALID


def test_other_bad_calls(lib):
    turn, bad = rope(), fa.FA_ERR_INVALID
    assert lib.fa_rotary_apply(None, turn, 0, None) == bad
    assert lib.fa_rotary_apply(struct(fa.FaRotaryRows, ROTATE), None, 0, None) == bad
    assert lib.fa_rotary_apply(struct(fa.FaRotaryRows, ROTATE), turn, 2, None) == bad
    own = rope(positions=at(9))
    packed = struct(fa.FaRotaryRows, ROTATE, cu_seqlens=at(8))
    assert lib.fa_rotary_apply(packed, own, 0, None) == bad
    assert lib.fa_paged_append(None, turn, None) == bad
    # queries, and an offset, where nothing turns them or the cache says where they are
    assert lib.fa_paged_append(struct(fa.FaPagedRows, APPEND), None, None) == bad
    shifted = rope(offset=1)
    assert lib.fa_paged_append(struct(fa.FaPagedRows, APPEND), shifted, None) == bad
    packed = struct(fa.FaPagedRows, APPEND, cu_seqlens=at(8), total=8, new_len=0)
    assert lib.fa_rotary_apply(struct(fa.FaRotaryRows, ROTATE), rope(offset=2 ** 31 - 7), 0,
                               None) == bad  # its last row's position
    strided = rope(positions=at(9), pos_stride=8)
    assert lib.fa_paged_append(packed, strided, None) == bad
    assert lib.fa_paged_keep(None, None) == bad


def test_good_calls_get_past_the_checks(lib):
    """Without a GPU the next thing that fails is the device."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")
    turn = rope()
    good = [dict(), dict(k=None, k_out=None, n_kv_heads=0), dict(q_out=at(0), k_out=at(1)),
            dict(q_out_stride=(4096, 128, 512)), dict(cu_seqlens=at(8)), dict(rows=0)]
    for kw in good:
        rows = struct(fa.FaRotaryRows, ROTATE, **kw)
        assert lib.fa_rotary_apply(rows, turn, 1, None) != fa.FA_ERR_INVALID, kw
    for kw in (dict(), dict(cu_seqlens=at(8), total=8, new_len=0)):
        rows = struct(fa.FaPagedRows, APPEND, **kw)
        assert lib.fa_paged_append(rows, turn, None) != fa.FA_ERR_INVALID, kw
    rows = struct(fa.FaPagedRows, APPEND, q=None, q_out=None, n_heads=0)
    assert lib.fa_paged_append(rows, None, None) != fa.FA_ERR_INVALID
    assert lib.fa_paged_keep(struct(fa.FaPagedKept, KEPT), None) != fa.FA_ERR_INVALID
    p = params()
    assert lib.fa_paged_tree_attention(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 64, FAKE, None, p,
                                       None) != fa.FA_ERR_INVALID


def test_structure_layouts():
    assert ctypes.sizeof(fa.FaRotary) == 40 and fa.FaRotary.scale.offset == 36
    assert ctypes.sizeof(fa.FaRotaryRows) == 160 and fa.FaRotaryRows.batch.offset == 136
    assert ctypes.sizeof(fa.FaPagedRows) == 184 and fa.FaPagedRows.batch.offset == 144
    assert ctypes.sizeof(fa.FaPagedKept) == 88 and fa.FaPagedKept.batch.offset == 56


def test_the_binding_refuses_what_it_cannot_pass_on():
    torch = pytest.importorskip("torch")
    P, Hk, ps, d = 4, 2, 16, 64
    c = [torch.zeros(P, Hk, ps, d, dtype=torch.bfloat16) for _ in range(2)]
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    x = torch.zeros(1, Hk, 3, d, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 3, d, dtype=torch.bfloat16)
    f = fa.rotary_inv_freq(32, device="cpu")[0]
    pos = torch.zeros(1, 3, dtype=torch.int32)
    mask = torch.ones(3, 3, dtype=torch.bool)
    keep, counts = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)

    def refused(text, call, *a, **kw):  # ("": for another reason than the device)
        with pytest.raises(ValueError, match=text or "^(?!.*CUDA device)"):
            call(*a, **kw)

    # all of it right but on the CPU
    refused("device", fa.rotary_fwd, q, x, f)
    refused("device", fa.rotary_bwd, q[0], x[0], f, cu_seqlens=cu)
    refused("device", fa.paged_cache_append, x, x, *c, table, lens, q=q, inv_freq=f, positions=pos)
    refused("device", fa.paged_cache_append, x[0], x[0], *c, table, lens, cu_seqlens=cu)
    refused("device", fa.paged_tree_attention, q, *c, table, lens, mask, scale=1.0)
    refused("device", fa.paged_cache_keep, *c, table, lens, keep, counts, 3)
    # rotations
    odd = torch.zeros(1, 4, 3, d + 4, dtype=torch.bfloat16)[..., :d]
    for y in (q.float(), odd, q.transpose(2, 3), q[0, 0]):
        refused("", fa.rotary_fwd, y, None, f)
    for y in (x[0], x[..., :32], x[:, :, :2], x.expand(2, Hk, 3, d), x.float()):
        refused("", fa.rotary_fwd, q, y, f)
    for y in (f.float(), f[None], f.repeat(2)[::2]):
        refused("inv_freq", fa.rotary_fwd, q, x, y)
    for y in (pos.long(), pos[:, :2], pos.expand(2, 3), pos[0, :2], torch.zeros(6, dtype=torch.int32)):
        refused("positions", fa.rotary_fwd, q, x, f, positions=y)
        refused("positions", fa.paged_cache_append, x, x, *c, table, lens, inv_freq=f, positions=y)
    refused("positions", fa.rotary_fwd, q[0], x[0], f, positions=pos)
    refused("contiguous", fa.rotary_fwd, q, x, f,
            positions=torch.zeros(1, 6, dtype=torch.int32)[:, ::2])
    refused("offset", fa.rotary_fwd, q, x, f, positions=pos, offset=1)
    for n in (2 ** 31, 2 ** 31 - 2, -2 ** 31 - 1):
        refused("32 bits", fa.rotary_fwd, q, x, f, offset=n)
    refused("cu_seqlens", fa.rotary_fwd, q, x, f, cu_seqlens=cu)
    refused("cu_seqlens", fa.rotary_fwd, q[0], x[0], f, cu_seqlens=cu, positions=pos[0])
    refused("cu_seqlens", fa.rotary_fwd, q[0], x[0], f, cu_seqlens=cu.long())
    refused("cu_seqlens", fa.rotary_fwd, q[0], x[0], f, cu_seqlens=cu[:1])
    # appends
    for y in (x.float(), x[:, :1], x.transpose(2, 3), x[0], x[..., :32], x.expand(2, Hk, 3, d)):
        refused("", fa.paged_cache_append, y, y, *c, table, lens)
    refused("shape", fa.paged_cache_append, x, x[:, :, :2], *c, table, lens)
    refused("inv_freq", fa.paged_cache_append, x, x, *c, table, lens, q=q)
    refused("inv_freq", fa.paged_cache_append, x, x, *c, table, lens, positions=pos)
    for y in (q[0], q[:, :, :2], q.float(), q.expand(2, 4, 3, d)):
        refused("", fa.paged_cache_append, x, x, *c, table, lens, q=y, inv_freq=f)
    # caches and indexes
    bad = [(c[0].float(), c[1]), (c[0][:, :1], c[1]), (c[0][0], c[1][0]),
           (c[0].transpose(1, 2).contiguous().transpose(1, 2), c[1])]
    for b in bad:
        refused("", fa.paged_cache_append, x, x, *b, table, lens)
        refused("", fa.paged_tree_attention, q, *b, table, lens, mask, scale=1.0)
        refused("", fa.paged_cache_keep, *b, table, lens, keep, counts, 3)
    for t, n in ((table.long(), lens), (table[0], lens), (table, lens.long()),
                 (table, lens.expand(2)), (table.expand(3, 2), lens)):
        refused("", fa.paged_cache_append, x, x, *c, t, n)
        refused("", fa.paged_tree_attention, q, *c, t, n, mask, scale=1.0)
        refused("", fa.paged_cache_keep, *c, t, n, keep, counts, 3)
    # trees
    for y in (q.float(), q[0], q[..., :32], q.expand(2, 4, 3, d), q.transpose(1, 2)):
        refused("", fa.paged_tree_attention, y, *c, table, lens, mask, scale=1.0)
    for y in (mask.float(), mask[:2], mask.expand(2, 3, 3), mask.t().contiguous().t()[:, :2],
              torch.ones(3, 6, dtype=torch.bool)[:, ::2], torch.ones(3, 3, dtype=torch.bool).t()):
        refused("", fa.paged_tree_attention, q, *c, table, lens, y, scale=1.0)
    for y, n in ((keep.long(), counts), (keep[0], counts), (keep.expand(2, 2), counts),
                 (torch.zeros(1, 4, dtype=torch.int32)[:, ::2], counts), (keep, counts.long())):
        refused("", fa.paged_cache_keep, *c, table, lens, y, n, 3)


def test_frequencies():
    torch = pytest.importorskip("torch")
    f, s = fa.rotary_inv_freq(64, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0
    np.testing.assert_allclose(f.numpy(), plain.inv_freq(64), rtol=1e-14)
    g, s = fa.rotary_inv_freq(64, factor=4.0, method="linear", device="cpu")
    np.testing.assert_allclose(g.numpy(), f.numpy() / 4, rtol=1e-14)
    g, s = fa.rotary_inv_freq(64, factor=4.0, method="base", device="cpu")
    assert g[0] == 1.0 and abs(g[-1] * 4 / f[-1] - 1) < 1e-12 and s == 1.0
    g, s = fa.rotary_inv_freq(64, 50000.0, factor=8.0, method="parts", original_len=4096, device="cpu")
    f = fa.rotary_inv_freq(64, 50000.0, device="cpu")[0]
    turns = f.numpy() * 4096 / (2 * math.pi)
    r = (g / f).numpy()
    assert (r[turns > 64] == 1).all() and np.allclose(r[turns < 0.5], 1 / 8)
    assert (np.diff(r) <= 0).all() and s == 0.1 * math.log(8) + 1
    for kw in (dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=64, factor=2.0),
               dict(rotary_dim=64, method="other"), dict(rotary_dim=64, base=0.0),
               dict(rotary_dim=64, factor=2.0, method="parts"),
               dict(rotary_dim=64, factor=float("inf"), method="linear")):
        with pytest.raises(ValueError):
            fa.rotary_inv_freq(**kw, device="cpu")


def test_plain_rotation_is_complex_multiplication():
    rng = np.random.default_rng(0)
    x, pos, f = rng.standard_normal((3, 5, 64)), rng.integers(0, 5000, (3, 5)), plain.inv_freq(32)
    z = np.exp(1j * pos[..., None] * f) * 1.5
    for inter in (False, True):
        a = x[..., 0:32:2] + 1j * x[..., 1:32:2] if inter else x[..., :16] + 1j * x[..., 16:32]
        y = plain.turn(x, pos, f, inter, 1.5)
        b = y[..., 0:32:2] + 1j * y[..., 1:32:2] if inter else y[..., :16] + 1j * y[..., 16:32]
        np.testing.assert_allclose(b, a * z, rtol=1e-9, atol=1e-11)
        np.testing.assert_array_equal(y[..., 32:], x[..., 32:])
        np.testing.assert_allclose(plain.turn(y, pos, f, inter, 1 / 1.5, True), x, atol=1e-12)


def test_plain_tree_attention_is_causal_for_a_chain():
    import oracle

    oracle.build()
    rng = np.random.default_rng(1)
    table, P = plain.make_table(rng, 2, 6)
    kc, vc = (rng.standard_normal((P, 2, 8, 64)).astype(np.float32) for _ in range(2))
    q, lengths = rng.standard_normal((2, 4, 5, 64)).astype(np.float32), np.array([33, 5])
    want = oracle.paged_fwd(q, kc, vc, table, lengths.astype(np.int32), scale=0.1, causal=True)
    got = plain.tree_attention(*(x.astype(np.float64) for x in (q, kc, vc)), table, lengths,
                               np.tril(np.ones((5, 5), bool)), 0.1)
    np.testing.assert_allclose(got[0], want[0], atol=1e-5)
    np.testing.assert_allclose(got[1], want[1], atol=1e-5)
