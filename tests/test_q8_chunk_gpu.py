"""Attention over the 8-bit cache with many query rows a kv head (chunks of a prompt), against the
paged oracle. The helpers and the tolerances are those of test_q8_cache_gpu.py; the weights here
have 11 bits, so that the 9 that the tolerance counts hold with room."""
import numpy as np
import pytest

from tests import q8_plain as plain
from tests.test_q8_cache_gpu import (A, _gpu, attend, bf16, check_attend, dev_cache,  # noqa: F401
                                     ints, make_attend, poison)

pytestmark = pytest.mark.gpu

CHUNKS = [
    A("rows32", 2, 4, 1, 8, 128, 16, 16, [300, 140]),  # the last in blocks of 16 rows
    A("rows33", 2, 3, 1, 11, 128, 16, 16, [300, 140]),
    A("rows34_d64", 2, 2, 2, 34, 64, 8, 2, [33, 1000]),
    A("rows40_d256", 1, 8, 1, 5, 256, 16, 16, [700]),
    A("rows48", 2, 4, 1, 12, 128, 16, 16, [12, 300]),
    A("rows49_d64", 2, 1, 1, 49, 64, 16, 4, [49, 130]),
    A("rows127", 1, 1, 1, 127, 128, 16, 16, [127]),
    A("rows128", 2, 8, 2, 32, 128, 16, 16, [500, 1290]),
    A("rows129_d64", 1, 3, 1, 43, 64, 32, 32, [1000]),
    A("rows150_page8_token_scales", 3, 6, 2, 50, 64, 8, 1, [49, 50, 700]),
    A("rows64_page256", 2, 8, 2, 16, 128, 256, 64, [400, 1029]),
    A("tile_edges", 6, 8, 2, 16, 128, 16, 16, [127, 128, 129, 255, 256, 257]),
    A("noncausal_rows256", 2, 4, 1, 64, 128, 16, 16, [1, 333], causal=False),
    A("noncausal_d64", 3, 2, 2, 70, 64, 16, 16, [0, 128, 200], causal=False),
    A("empty_among", 4, 4, 1, 16, 128, 16, 16, [0, 90, 0, 16]),
    A("all_empty", 2, 4, 1, 20, 64, 16, 16, [0, 0]),
    A("past_their_length", 3, 2, 1, 200, 128, 16, 16, [1, 130, 199]),
    A("whole_prompt", 1, 2, 2, 512, 128, 16, 16, [512]),
    A("split_over_many", 1, 4, 1, 16, 128, 64, 64, [20_000]),
    A("split_d64", 2, 4, 1, 20, 64, 16, 16, [9000, 3]),
    A("many_short", 60, 4, 1, 12, 64, 16, 16, [(i * 37) % 200 for i in range(60)]),
    A("long_rows", 1, 2, 1, 300, 128, 16, 16, [3001]),
]


@pytest.mark.parametrize("c", CHUNKS, ids=lambda c: c["name"])
def test_chunk_matches_the_oracle(c):
    import flash_attention_gb300 as fa

    _, table, P, cache, q = make_attend(c)
    cache = poison(c, table, cache)
    qt, q = bf16(q)
    o, lse = attend(c, table, dev_cache(*cache), qt)
    assert fa.fa_device_status(True) == fa.FA_OK
    print(c["name"], check_attend(c, table, cache, q, o, lse))


@pytest.mark.parametrize("name", ["sink", "scales", "tiny", "large", "rising"])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_with_uneven_softmax_and_scales(name, d):
    """A key that takes nearly all of the weight with thousands of small ones behind it; value
    scales over 2^40; tiny and large queries; scores that rise from tile to tile."""
    import flash_attention_gb300 as fa

    c = A(name, 2, 4, 2, 32, d, 16, 1, [3000, 4500])
    rng, table, P, cache, q = make_attend(c)
    if name == "sink":
        q[:] = 1.0
        for b in range(2):
            cache[0][table[b, 3], :, 5] = plain.to_code(np.full(d, 24.0))
            cache[2][table[b, 3], :, 5] = 2.0 ** -4 * (128 / d) ** 0.5
        cache[0][:] = np.where(np.arange(16)[:, None] % 16 == 5, cache[0],
                               plain.to_code(plain.VALUES[cache[0]] / 64))
        cache[1][:] = plain.to_code(np.abs(plain.VALUES[cache[1]]))
        for b in range(2):
            cache[1][table[b, 3], :, 5] = plain.to_code(2.0 ** -9)
    elif name == "scales":
        cache[3][:] = 2.0 ** rng.integers(-30, 10, cache[3].shape)
    elif name == "tiny":
        q *= 1e-30
    elif name == "large":
        q *= 30
    else:
        q[:] = 1.0
        for b in range(2):
            j = np.arange(c["lengths"][b])
            at, slot = table[b, j // 16], j % 16
            cache[0][at, :, slot] = plain.to_code(1 + 0 * cache[0][at, :, slot])
            cache[2][at, :, slot] = (j / 300.0)[:, None]
    qt, q = bf16(q)
    o, lse = attend(c, table, dev_cache(*cache), qt)
    assert fa.fa_device_status(True) == fa.FA_OK
    print(name, check_attend(c, table, cache, q, o, lse))


@pytest.mark.parametrize("d,H,lq", [(128, 8, 20), (64, 2, 90)])
def test_chunk_nan_behind_a_row_does_not_reach_it(d, H, lq):
    """NaN in keys and values that only the later of the new positions see."""
    import torch

    c = A("hidden", 2, H, 2, lq, d, 16, 16, [300, 129])
    _, table, P, cache, q = make_attend(c)
    qt, _ = bf16(q)
    o0, l0 = attend(c, table, dev_cache(*cache), qt)
    for which in (0, 1):
        bad = [x.copy() for x in cache]
        for b, n in enumerate(c["lengths"]):  # the last position, and the one two before it
            bad[which][table[b, (n - 1) // 16], 1, (n - 1) % 16, 5] = 0x7F
            bad[which][table[b, (n - 3) // 16], 0, (n - 3) % 16, 9:12] = 0xFF
        o, lse = attend(c, table, dev_cache(*bad), qt)
        sees = torch.zeros(2, H, lq, dtype=torch.bool, device="cuda")
        sees[:, H // 2:, lq - 1] = True
        sees[:, :H // 2, lq - 3:] = True
        assert torch.equal(o[~sees], o0[~sees]) and torch.equal(lse[~sees], l0[~sees])
        if which == 0:
            assert o[sees].isnan().all() and lse[sees].isnan().all()
        else:
            assert torch.equal(lse, l0)
            assert o[:, H // 2:, lq - 1, 5].isnan().all()
            assert o[:, :H // 2, lq - 3:, 9:12].isnan().all()


def test_chunk_nan_stays_in_its_rows():
    import torch

    c = A("nan", 2, 8, 2, 16, 128, 16, 16, [300, 200])
    _, table, P, cache, q = make_attend(c)
    qt, _ = bf16(q)
    o0, l0 = attend(c, table, dev_cache(*cache), qt)
    bad = qt.clone()
    bad[0, 1, 3, 7] = float("nan")
    bad[1, 6, 15, 9] = float("inf")
    o, lse = attend(c, table, dev_cache(*cache), bad)
    hit = torch.zeros(2, 8, 16, dtype=torch.bool, device="cuda")
    hit[0, 1, 3] = hit[1, 6, 15] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(o[~hit], o0[~hit]) and torch.equal(lse[~hit], l0[~hit])
    cache[1][table[1, 2], 1, 3, 5] = 0x7F  # a value that all rows of sequence 1, kv head 1 see
    o, lse = attend(c, table, dev_cache(*cache), qt)
    hit = torch.zeros(2, 8, 16, 128, dtype=torch.bool, device="cuda")
    hit[1, 4:, :, 5] = True
    assert torch.equal(o.isnan(), hit) and torch.equal(lse, l0)


def test_chunk_out_of_range_inputs_are_flagged_not_faulted():
    import torch

    import flash_attention_gb300 as fa

    c = A("bad", 2, 4, 2, 40, 128, 16, 16, [50, 100])
    _, table, P, cache, q = make_attend(c)
    qt, q64 = bf16(q)
    got = dev_cache(*cache)
    attend(dict(c, lengths=[5000, 100]), table, got, qt)  # clamped to the table's capacity
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    attend(dict(c, lengths=[-4, 100]), table, got, qt)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    t = table.copy()
    t[1, 0], t[1, 1] = P + 7, -3  # pages outside the cache read as zero keys and values
    o, lse = attend(c, t, got, qt)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    zero = [np.concatenate([x, np.zeros_like(x[:1]) + (i > 1)]) for i, x in enumerate(cache)]
    t[1, 0] = t[1, 1] = P
    check_attend(c, t, zero, q64, o, lse)
    o, lse = attend(c, table, got, qt)
    assert fa.fa_device_status(True) == fa.FA_OK and torch.isfinite(o.float()).all()


def test_chunk_writes_its_outputs_and_nothing_else():
    """o and lse inside filled buffers, through the C ABI, for whole and cut units."""
    import ctypes

    import torch

    import flash_attention_gb300 as fa

    for d, lq, lengths in ((64, 37, [5, 0, 900]), (128, 13, [9000, 1, 0])):
        c = A("guard", 3, 8, 2, lq, d, 16, 16, lengths)
        _, table, P, cache, q = make_attend(c)
        got, (qt, q64) = dev_cache(*cache), bf16(q)
        n, m, pad = qt.numel(), 3 * 8 * lq, 512
        for with_lse in (True, False):
            o = torch.full((n + 2 * pad,), -7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((m + 2 * pad,), -7.0, device="cuda")
            tb, ln = ints(table), ints(lengths)
            s = fa._q8_cache(*got, torch)
            p = fa.FaPagedParams(3, 8, 2, lq, d, 16, table.shape[1], P, d ** -0.5, 1, 0, 0)
            rc = fa.load_library().fa_q8_paged_attention(
                qt.data_ptr(), ctypes.byref(s), tb.data_ptr(), ln.data_ptr(),
                o.data_ptr() + 2 * pad, lse.data_ptr() + 4 * pad if with_lse else None,
                ctypes.byref(p), torch.cuda.current_stream().cuda_stream)
            assert rc == fa.FA_OK and fa.fa_device_status(True) == fa.FA_OK
            for x in (o, lse):
                assert (x[:pad] == -7).all() and (x[-pad:] == -7).all()
            inner = lse[pad:-pad].view(3, 8, lq)
            if with_lse:
                check_attend(c, table, cache, q64, o[pad:-pad].view(qt.shape), inner)
            else:
                assert (inner == -7).all()


def test_chunk_is_reproducible_and_captured():
    """The same bits again, on another stream, and from a captured graph whose inputs change."""
    import torch

    import flash_attention_gb300 as fa

    c = A("again", 3, 8, 2, 24, 128, 16, 16, [3000, 70, 900])
    _, table, P, cache, q = make_attend(c)
    got, (qt, q64) = dev_cache(*cache), bf16(q)
    o0, l0 = attend(c, table, got, qt)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        o, lse = attend(c, table, got, qt, stream=s)
        s.synchronize()
        assert torch.equal(o, o0) and torch.equal(lse, l0)
    tb, ln, qc = ints(table), ints(c["lengths"]), torch.zeros_like(qt)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og, lg = fa.q8_paged_attention(qc, *got, tb, ln, scale=c["d"] ** -0.5)
    for lengths in (c["lengths"], [24, 0, 1000]):
        ln.copy_(ints(lengths))
        qc.copy_(qt)
        g.replay()
        torch.cuda.synchronize()
        check_attend(dict(c, lengths=lengths), table, cache, q64, og, lg)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_chunk_waits_that_run_out_are_reported():
    import flash_attention_gb300 as fa

    for d in (64, 128):
        c = A("long", 2, 8, 2, 16, d, 16, 16, [5000, 300])
        _, table, P, cache, q = make_attend(c)
        got, (qt, q64) = dev_cache(*cache), bf16(q)
        try:
            fa.fa_set_wait_limit_ns(1)
            attend(c, table, got, qt)
            assert fa.fa_device_status(True) == fa.FA_ERR_DEVICE_TIMEOUT
        finally:
            fa.fa_set_wait_limit_ns(0)
        o, lse = attend(c, table, got, qt)
        assert fa.fa_device_status(True) == fa.FA_OK
        check_attend(c, table, cache, q64, o, lse)
