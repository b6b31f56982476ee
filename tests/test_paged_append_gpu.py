"""Appending to the paged bf16 cache with the rotation on the way, and keeping accepted nodes, on the
GPU against plain 64-bit forms. What is copied has to be the same bits; what is turned is held to
tests.draft_plain.turn_bound."""
import numpy as np
import pytest

from tests import draft_plain as plain
from tests.test_rotary_gpu import _gpu, bf16, freqs, ints, laid_out  # noqa: F401

pytestmark = pytest.mark.gpu

APPENDS = [
    # name, H, Hk, d, rot, page, lengths before, new rows of each sequence
    ("one_token", 8, 2, 128, 128, 16, [0, 1, 15, 16, 37], [1] * 5),
    ("one_token_d64_part", 3, 3, 64, 16, 64, [0, 31, 63, 100], [1] * 4),
    ("one_token_d256", 4, 1, 256, 256, 8, [0, 7, 8, 9], [1] * 4),
    ("five_tokens", 2, 2, 128, 32, 32, [0, 29, 30, 31, 64], [5] * 5),
    ("ragged", 8, 2, 128, 64, 16, [0, 3, 0, 50, 16], [33, 0, 1, 17, 300]),
    ("ragged_d64", 2, 2, 64, 64, 8, [5, 0, 0], [1, 70, 129]),
    ("ragged_d256_page256", 2, 1, 256, 128, 256, [0, 255, 256, 300], [5, 3, 700, 1]),
    ("many_sequences", 1, 1, 64, 32, 16, [0] * 70, list(range(70))),
]


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("layout", ["heads", "rows", "fused"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: c[0])
def test_append_matches_the_definition(case, layout, inter):
    import flash_attention_gb300 as fa

    name, H, Hk, d, rot, ps, past, new = case
    rng = np.random.default_rng(len(name) + d)
    B, total = len(past), sum(new)
    lengths = np.array(past) + new
    per = int(-(-lengths.max() // ps)) + 1
    table, P = plain.make_table(rng, B, per)
    (kc, kcx), (vc, vcx) = (bf16(rng.standard_normal((P, Hk, ps, d))) for _ in range(2))
    fixed = len(set(new)) == 1
    cu = np.concatenate([[0], np.cumsum(new)])
    own = rng.integers(0, 3000000, total)

    def rows(heads):
        if fixed:
            return laid_out(rng.standard_normal((B, heads, new[0], d)), layout)
        return laid_out(rng.standard_normal((heads, total, d)), layout)

    (k, kx), (v, vx), (q, qx) = rows(Hk), rows(Hk), rows(H)
    freq = plain.inv_freq(rot)

    def seq(x, b):
        return x[b] if fixed else x[:, cu[b]:cu[b + 1]]

    for kind in ("places", "positions", "no rotation"):
        kc2, vc2 = kc.clone(), vc.clone()
        kw = {} if fixed else dict(cu_seqlens=ints(cu))
        scale = 1.0
        if kind == "positions":
            scale = 1.25
            pos = [own[cu[b]:cu[b + 1]] for b in range(B)]
            kw["positions"] = ints(own.reshape(B, -1) if fixed else own)
        else:
            pos = [np.arange(length - n, length) for length, n in zip(lengths, new)]
        if kind == "no rotation":
            assert fa.paged_cache_append(k, v, kc2, vc2, ints(table), ints(lengths), **kw) is None
            turned = [seq(kx, b) for b in range(B)]
            slack = [np.zeros_like(t) for t in turned]
        else:
            qo = fa.paged_cache_append(k, v, kc2, vc2, ints(table), ints(lengths), q=q,
                                       inv_freq=freqs(freq), interleaved=inter, rotary_scale=scale,
                                       **kw)
            turned = [plain.turn(seq(kx, b), pos[b], freq, inter, scale) for b in range(B)]
            slack = [plain.turn_bound(seq(kx, b), turned[b], rot, inter, scale) for b in range(B)]
            assert qo.is_contiguous() and qo.shape == q.shape
            for b in range(B):
                want = plain.turn(seq(qx, b), pos[b], freq, inter, scale)
                err = np.abs(seq(qo.double().cpu().numpy(), b) - want)
                assert (err <= plain.turn_bound(seq(qx, b), want, rot, inter, scale)).all()
            for x in slack:
                x[..., rot:] = 0
        wk, wv, bound = kcx.copy(), vcx.copy(), np.zeros_like(kcx)
        plain.append(wk, wv, turned, [seq(vx, b) for b in range(B)], table, lengths)
        plain.append(bound, bound.copy(), slack, slack, table, lengths)
        assert (np.abs(kc2.double().cpu().numpy() - wk) <= bound).all()
        np.testing.assert_array_equal(vc2.double().cpu().numpy(), wv)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_one_position_for_all_sequences():
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(2)
    k, _ = bf16(rng.standard_normal((3, 2, 4, 64)))
    kc = torch.zeros(3, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    outs = []
    for pos in (np.array([5, 6, 6, 7]), np.tile([5, 6, 6, 7], (3, 1))):
        a, b = kc.clone(), kc.clone()
        fa.paged_cache_append(k, k, a, b, ints([[0], [1], [2]]), ints([4, 4, 4]),
                              inv_freq=freqs(plain.inv_freq(64)), positions=ints(pos))
        outs.append((a, b))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1][:, :, :4], k)


def test_rows_that_have_no_place_are_left_out():
    """Padded entries (length 0), rows before position 0, lengths and pages out of range: the rest is
    written, nothing else is touched, and what is out of range is reported."""
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(6)
    B, Hk, n, d, ps, per = 6, 2, 4, 64, 8, 2
    lengths = np.array([0, 2, 10, 17, -3, 12])
    table, P = plain.make_table(rng, B, per)
    table[5, 1] = P
    (kc, kcx), (vc, vcx) = (bf16(rng.standard_normal((P, Hk, ps, d))) for _ in range(2))
    (k, kx), (v, vx) = (bf16(rng.standard_normal((B, Hk, n, d))) for _ in range(2))
    q, qx = bf16(rng.standard_normal((B, 4, n, d)))
    freq = plain.inv_freq(32)
    for bad in (False, True):
        live = slice(0, B) if bad else slice(0, 3)
        kc2, vc2 = kc.clone(), vc.clone()
        qo = fa.paged_cache_append(k[live], v[live], kc2, vc2, ints(table[live]),
                                   ints(lengths[live]), q=q[live], inv_freq=freqs(freq))
        wk, wv = kcx.copy(), vcx.copy()
        turned = [plain.turn(kx[b], lengths[b] - n + np.arange(n), freq) for b in range(B)][live]
        plain.append(wk, wv, turned, list(vx[live]), table[live], lengths[live])
        assert np.abs(kc2.double().cpu().numpy() - wk).max() <= 2 ** -7 * np.abs(wk).max()
        np.testing.assert_array_equal(kc2.double().cpu().numpy()[wk == kcx], wk[wk == kcx])
        np.testing.assert_array_equal(vc2.double().cpu().numpy(), wv)
        pos = (lengths[:, None] - n + np.arange(n))[live]
        want = plain.turn(qx[live], pos[:, None], freq)
        assert (np.abs(qo.double().cpu().numpy() - want)
                <= plain.turn_bound(qx[live], want, 32, False, 1.0)).all()
        assert fa.fa_device_status(True) == (fa.FA_ERR_BAD_INPUT if bad else fa.FA_OK)


def test_packed_rows_behind_the_last_sequence_and_bad_offsets():
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(7)
    k, kx = bf16(rng.standard_normal((1, 12, 64)))
    kc0 = torch.full((4, 1, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    table = ints([[0, 1], [2, 3]])
    kc, vc = kc0.clone(), kc0.clone()
    fa.paged_cache_append(k, k, kc, vc, table, ints([6, 3]), cu_seqlens=ints([0, 6, 9]))
    assert torch.equal(vc[0, :, :6], k[:, :6]) and torch.equal(vc[2, :, :3], k[:, 6:9])
    assert (vc[0, :, 6:] == 7).all() and (vc[2, :, 3:] == 7).all() and (vc[[1, 3]] == 7).all()
    assert torch.equal(kc, vc) and fa.fa_device_status(True) == fa.FA_OK
    for cu in ([0, 6, 13], [0, 8, 6], [2, 6, 9], [-4, 6, 9]):
        fa.paged_cache_append(k, k, kc0.clone(), kc0.clone(), table, ints([6, 3]), cu_seqlens=ints(cu))
        assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT, cu


def test_a_cache_past_32_bits():
    """Pages behind 2^31 elements, of both caches."""
    import torch

    import flash_attention_gb300 as fa

    Hk, ps, d = 8, 256, 128
    P = (1 << 31) // (Hk * ps * d) + 8
    kc = torch.zeros(P, Hk, ps, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rng = np.random.default_rng(1)
    k, _ = bf16(rng.standard_normal((1, Hk, 20, d)))
    table = ints([[3, P - 1]])
    fa.paged_cache_append(k, k, kc, vc, table, ints([ps + 10]))
    for x in (kc, vc):
        assert torch.equal(x[3, :, -10:], k[0, :, :10]) and torch.equal(x[P - 1, :, :10], k[0, :, 10:])
    keep = ints([[0, 3, 10, 12, 19]])
    new = fa.paged_cache_keep(kc, vc, table, ints([ps + 10]), keep, ints([5]), 20)
    assert new.tolist() == [ps - 5]
    for x in (kc, vc):
        assert torch.equal(x[3, :, -10:-5], k[0][:, [0, 3, 10, 12, 19]])


KEEPS = [  # Hk, d, page, T, M, lengths
    (2, 128, 16, 8, 8, [8, 9, 40, 33]), (1, 64, 8, 256, 256, [256, 300, 511]),
    (8, 128, 32, 17, 5, [17, 100, 31, 32, 1000]), (3, 256, 8, 1, 1, [1, 2, 9]),
    (1, 64, 128, 64, 40, [64] * 33),
]


@pytest.mark.parametrize("case", KEEPS, ids=str)
def test_keep_moves_the_accepted_rows(case):
    import flash_attention_gb300 as fa

    Hk, d, ps, T, M, lengths = case
    rng = np.random.default_rng(T + M)
    B = len(lengths)
    table, P = plain.make_table(rng, B, -(-max(lengths) // ps) + 1)
    (kc, kcx), (vc, vcx) = (bf16(rng.standard_normal((P, Hk, ps, d))) for _ in range(2))
    for case in range(3):
        counts = rng.integers(0, M + 1, B) if case else np.full(B, M)
        keep = np.stack([np.sort(rng.permutation(T)[:M]) for _ in range(B)])
        if case == 2:
            keep[:] = np.arange(M)  # a chain: nothing moves
        rows = keep.copy()
        for b in range(B):
            rows[b, counts[b]:] = -99  # behind the count: any
        kc2, vc2 = kc.clone(), vc.clone()
        new = fa.paged_cache_keep(kc2, vc2, ints(table), ints(lengths), ints(rows), ints(counts), T)
        wk, wv = kcx.copy(), vcx.copy()
        kept = [list(keep[b, :counts[b]]) for b in range(B)]
        assert new.tolist() == plain.keep((wk, wv), table, lengths, kept, T)
        np.testing.assert_array_equal(kc2.double().cpu().numpy(), wk)
        np.testing.assert_array_equal(vc2.double().cpu().numpy(), wv)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_keep_of_short_trees_and_padded_entries():
    """A tree of three nodes at the end of eight, of a sequence of five keys: the columns before it keep
    their places, some of them before the sequence's start. A padded entry has length 0 and count 0."""
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(3)
    kc, _ = bf16(rng.standard_normal((4, 2, 8, 64)))
    old, vc = kc.clone(), kc.clone()
    keep = ints([[0, 1, 2, 3, 4, 6, 7, 0], [0] * 8])
    new = fa.paged_cache_keep(kc, vc, ints([[2], [0]]), ints([5, 0]), keep, ints([7, 0]), 8)
    assert new.tolist() == [4, 0] and torch.equal(kc, vc)
    assert torch.equal(kc[2, :, [2, 3]], old[2, :, [3, 4]]) and torch.equal(kc[2, :, :2], old[2, :, :2])
    kc[2], old[2] = 0, 0
    assert torch.equal(kc, old) and fa.fa_device_status(True) == fa.FA_OK


def test_keep_leaves_sequences_with_bad_nodes_alone():
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(4)
    kc, _ = bf16(rng.standard_normal((4, 1, 8, 64)))
    bad = [([3, 2], 2, 8), ([3, 3], 2, 8), ([-1, 2], 2, 8), ([1, 4], 2, 8), ([1, 2], 3, 8),
           ([1, 2], -1, 8), ([1, 2], 2, 17), ([1, 2], 2, -1), ([1, 3], 2, 3),
           ([1, 2147483647], 2, 8), ([-2147483648, 1], 2, 8)]
    for nodes, count, length in bad:
        a, b = kc.clone(), kc.clone()
        new = fa.paged_cache_keep(a, b, ints([[1, 2], [3, 0]]), ints([length, 8]),
                                  ints([nodes, [1, 3]]), ints([count, 2]), 4)
        assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT, (nodes, count, length)
        assert new.tolist() == [length, 6] and torch.equal(a, b) and torch.equal(a[:3], kc[:3])
        assert torch.equal(a[3, :, [4, 5]], kc[3, :, [5, 7]])
    # a page outside the cache: its rows stay out
    a, b = kc.clone(), kc.clone()
    new = fa.paged_cache_keep(a, b, ints([[1, 4]]), ints([10]), ints([[1, 3]]), ints([2]), 4)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT and new.tolist() == [8]
    want = kc.clone()
    want[1, :, 6] = kc[1, :, 7]
    assert torch.equal(a, want) and torch.equal(b, want)


def test_captured_and_on_another_stream():
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(5)
    (k, _), (q, _) = bf16(rng.standard_normal((2, 2, 6, 128))), bf16(rng.standard_normal((2, 4, 6, 128)))
    table, lens, f = ints([[0, 1], [2, 3]]), ints([12, 6]), freqs(plain.inv_freq(128))
    keep, counts = ints([[1, 4], [0, 5]]), ints([2, 2])

    def step(kc, vc, **kw):
        qo = fa.paged_cache_append(k, k, kc, vc, table, lens, q=q, inv_freq=f, **kw)
        return qo, fa.paged_cache_keep(kc, vc, table, lens, keep, counts, 6, **kw)

    new = lambda: torch.zeros(4, 2, 8, 128, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    kc, vc = new(), new()
    want = step(kc, vc)
    s, kc2, vc2 = torch.cuda.Stream(), new(), new()
    s.wait_stream(torch.cuda.current_stream())
    got = step(kc2, vc2, stream=s)
    s.synchronize()
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and all(map(torch.equal, got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(kc2, vc2)
    k.mul_(2)
    kc.zero_(), kc2.zero_(), vc2.zero_(), vc.zero_()
    graph.replay()
    want = step(kc, vc)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and all(map(torch.equal, got, want))
