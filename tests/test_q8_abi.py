"""The 8-bit cache's entry points without a GPU: every bad argument is refused before the device or
any pointer is touched, and the binding's own checks."""
import ctypes

import pytest

import flash_attention_gb300 as fa

FAKE = 0x100000  # aligned, never dereferenced: checks come first

CACHE = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=10, n_kv_heads=2,
             page_size=16, head_dim=128, scale_block=16, reserved=0)
ROWS = dict(k=FAKE, v=FAKE, k_stride=(512, 256, 128), v_stride=(512, 256, 128), cu_seqlens=FAKE,
            block_table=FAKE, lengths=FAKE, batch=2, max_pages=4, total=8, new_len=0)
PARAMS = dict(batch=2, n_heads=8, n_kv_heads=2, q_len=1, head_dim=128, page_size=16, max_pages=4,
              num_pages=10, scale=0.1, causal=1, num_splits=0, reserved=0)

BAD_CACHE = [dict(k=None), dict(v=FAKE + 8), dict(k_scale=None), dict(v_scale=FAKE + 2),
             dict(num_pages=0), dict(num_pages=1 << 30), dict(n_kv_heads=0), dict(page_size=12),
             dict(page_size=4), dict(page_size=512), dict(head_dim=96), dict(scale_block=0),
             dict(scale_block=32), dict(scale_block=12), dict(reserved=1)]
BAD_ROWS = [dict(k=None), dict(v=FAKE + 8), dict(k_stride=(512, 256, 127)),
            dict(v_stride=(-8, 256, 128)), dict(cu_seqlens=FAKE + 2), dict(block_table=None),
            dict(block_table=FAKE + 1), dict(batch=0), dict(max_pages=0), dict(max_pages=1 << 19),
            dict(total=-1), dict(new_len=3), dict(cu_seqlens=None),
            dict(total=(1 << 31) - 1, batch=1 << 30)]
BAD_WRITE = [dict(lengths=None), dict(lengths=FAKE + 2),
             dict(cu_seqlens=None, total=0, new_len=0),
             dict(cu_seqlens=None, total=0, new_len=1 << 23),
             dict(cu_seqlens=None, total=0, new_len=1 << 22, batch=1 << 20)]
BAD_READ = [dict(), dict(lengths=None, cu_seqlens=None, total=0, new_len=3),
            dict(lengths=None, k_stride=(0, 1024, 0)), dict(lengths=None, v_stride=(0, 64, 256))]


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load_library()


def cache(**kw):
    return fa.FaQ8Cache(**dict(CACHE, **kw))


def rows(**kw):
    d = dict(ROWS, **kw)
    for n in ("k_stride", "v_stride"):
        d[n] = (ctypes.c_int64 * 3)(*d[n])
    return fa.FaQ8Rows(**d)


def ids(kw):
    return ",".join(f"{k}={v}" for k, v in kw.items()) or "lengths given"


@pytest.mark.parametrize("kw", BAD_CACHE, ids=ids)
def test_bad_caches_are_refused(lib, kw):
    c = cache(**kw)
    assert lib.fa_q8_cache_write(c, rows(), None) == fa.FA_ERR_INVALID
    assert lib.fa_q8_cache_read(c, rows(lengths=None), None) == fa.FA_ERR_INVALID
    p = fa.FaPagedParams(**PARAMS)
    assert lib.fa_q8_paged_attention(FAKE, c, FAKE, FAKE, FAKE, None, p, None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", BAD_ROWS + BAD_WRITE, ids=ids)
def test_bad_writes_are_refused(lib, kw):
    assert lib.fa_q8_cache_write(cache(), rows(**kw), None) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(lengths=None, **k) for k in BAD_ROWS] + BAD_READ, ids=ids)
def test_bad_reads_are_refused(lib, kw):
    assert lib.fa_q8_cache_read(cache(), rows(**kw), None) == fa.FA_ERR_INVALID


def test_null_structures_are_refused(lib):
    assert lib.fa_q8_cache_write(None, rows(), None) == fa.FA_ERR_INVALID
    assert lib.fa_q8_cache_write(cache(), None, None) == fa.FA_ERR_INVALID
    assert lib.fa_q8_cache_read(cache(), None, None) == fa.FA_ERR_INVALID
    assert lib.fa_q8_paged_attention(FAKE, None, FAKE, FAKE, FAKE, None,
                                     fa.FaPagedParams(**PARAMS), None) == fa.FA_ERR_INVALID
    assert lib.fa_q8_paged_attention(FAKE, cache(), FAKE, FAKE, FAKE, None, None, None) == \
        fa.FA_ERR_INVALID


BAD_PARAMS = [dict(batch=0), dict(n_heads=7), dict(q_len=0), dict(scale=0.0), dict(causal=2),
              dict(num_splits=1), dict(num_splits=-1), dict(reserved=1), dict(n_kv_heads=4),
              dict(head_dim=64), dict(page_size=32), dict(num_pages=9), dict(max_pages=0),
              dict(max_pages=1 << 19), dict(batch=40000), dict(q_len=1 << 23)]


@pytest.mark.parametrize("kw", BAD_PARAMS, ids=ids)
def test_bad_attention_parameters_are_refused(lib, kw):
    p = fa.FaPagedParams(**dict(PARAMS, **kw))
    assert lib.fa_q8_paged_attention(FAKE, cache(), FAKE, FAKE, FAKE, None, p, None) == \
        fa.FA_ERR_INVALID


@pytest.mark.parametrize("at,value", [(0, None), (0, FAKE + 8), (2, None), (3, FAKE + 2),
                                      (4, None), (5, FAKE + 1)])
def test_bad_attention_pointers_are_refused(lib, at, value):
    args = [FAKE, cache(), FAKE, FAKE, FAKE, None]
    args[at] = value
    assert lib.fa_q8_paged_attention(*args, fa.FaPagedParams(**PARAMS), None) == fa.FA_ERR_INVALID


def test_structure_layouts():
    assert ctypes.sizeof(fa.FaQ8Cache) == 56 and fa.FaQ8Cache.num_pages.offset == 32
    assert ctypes.sizeof(fa.FaQ8Rows) == 104 and fa.FaQ8Rows.cu_seqlens.offset == 64
    assert fa.FaQ8Rows.batch.offset == 88


def test_the_binding_refuses_what_it_cannot_pass_on():
    torch = pytest.importorskip("torch")
    P, Hk, ps, d = 4, 2, 16, 64
    c = fa.make_q8_cache(P, Hk, ps, d, 8, device="cpu")
    assert c[0].dtype == torch.float8_e4m3fn and c[2].shape == (P, Hk, 2)
    with pytest.raises(ValueError):
        fa.make_q8_cache(P, Hk, ps, d, 12, device="cpu")
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    x = torch.zeros(1, Hk, 1, d, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 1, d, dtype=torch.bfloat16)

    def refused(text, call, *a, **kw):
        with pytest.raises(ValueError, match=text):
            call(*a, **kw)

    # all of it right but on the CPU
    refused("device", fa.q8_cache_write, x, x, *c, table, lens)
    refused("device", fa.q8_cache_write, x[0], x[0], *c, table, lens, cu_seqlens=cu)
    refused("device", fa.q8_cache_read, *c, table, cu, 1)
    refused("device", fa.q8_paged_attention, q, *c, table, lens, scale=1.0)
    # the cache
    bad = [(c[0].float(), *c[1:]), (c[0][:, :1], *c[1:]), (c[0], c[1], c[2].double(), c[3]),
           (c[0], c[1], c[2][:, :, :1], c[3]), (c[0], c[1], c[2][:3], c[3][:3]),
           (c[0].transpose(1, 2).contiguous().transpose(1, 2), *c[1:])]
    for b in bad:
        refused("", fa.q8_paged_attention, q, *b, table, lens, scale=1.0)
        refused("", fa.q8_cache_read, *b, table, cu, 1)
        refused("", fa.q8_cache_write, x, x, *b, table, lens)
    # rows
    odd = torch.zeros(1, Hk, 1, d + 4, dtype=torch.bfloat16)[..., :d]
    for y in (x.float(), x[:, :1], x.transpose(2, 3), odd, x[0], x[..., :32],
              x.expand(2, Hk, 1, d)):
        refused("", fa.q8_cache_write, y, y, *c, table, lens)
    refused("shape", fa.q8_cache_write, x, x.expand(1, Hk, 2, d), *c, table, lens)
    # indexes and queries
    for t, n in ((table.long(), lens), (table[0], lens), (table, lens.long()),
                 (table, lens.expand(2)), (table.expand(3, 2), lens)):
        refused("", fa.q8_cache_write, x, x, *c, t, n)
        refused("", fa.q8_paged_attention, q, *c, t, n, scale=1.0)
    refused("cu_seqlens", fa.q8_cache_read, *c, table, torch.zeros(3, dtype=torch.int32), 1)
    for y in (q.float(), q[0], q[..., :32], q.expand(1, 4, 2, d), q.expand(2, 4, 1, d)):
        refused("", fa.q8_paged_attention, y, *c, table, lens, scale=1.0)
