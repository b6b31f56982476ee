"""Attention of trees of drafted tokens over the paged cache on the GPU against the plain 64-bit form.

Tolerances, per element: O is rounded to bf16 (2^-8 of |o|) and each softmax weight too (2^-8 of
itself, against sum_j p_j |v_j|); the 32-bit arithmetic between (sums of up to 2^14 terms, exponentials
good to 2^-22, scores of at most 2^6 in base 2 rounded to 2^-24 of themselves) stays below 2^-14 of the
same sum. L: the 32-bit score and sum, below 2^-17 of max(1, |L|) by the same count."""
import numpy as np
import pytest

from tests import draft_plain as plain
from tests.test_rotary_gpu import _gpu, bf16, ints  # noqa: F401

pytestmark = pytest.mark.gpu


def check(got, want, rows=slice(None)):
    o, lse = (t.double().cpu().numpy()[rows] for t in got)
    wo, wl, w = (x[rows] for x in want)
    np.testing.assert_array_equal(np.isnan(o), np.isnan(wo))
    inf = np.isinf(wo)
    np.testing.assert_array_equal(o[inf], wo[inf])
    fine = np.isfinite(wo)
    err = np.abs(o[fine] - wo[fine])
    bound = (2.0 ** -8 * np.abs(wo) + (2.0 ** -8 + 2.0 ** -14) * w)[fine]
    assert (err <= bound + 1e-30).all(), (err.max(), (err / (bound + 1e-30)).max())
    none = np.isneginf(wl)
    assert (lse[none] == -np.inf).all() and (o[none] == 0).all()
    wl, lse = wl[~none], lse[~none]
    np.testing.assert_array_equal(np.isnan(lse), np.isnan(wl))
    ok = np.isfinite(wl)
    assert (np.abs(lse - wl)[ok] <= 2.0 ** -17 * np.maximum(1, np.abs(wl[ok]))).all()


def make(seed, B, H, Hk, T, d, ps, lengths, spare=3, extra=1):
    rng = np.random.default_rng(seed)
    table, P = plain.make_table(rng, B, -(-max(max(lengths), 1) // ps) + extra, spare)
    kc, vc = (bf16(rng.standard_normal((P, Hk, ps, d))) for _ in range(2))
    q = bf16(rng.standard_normal((B, H, T, d)))
    return rng, table, kc, vc, q


def masks(rng, B, T, kind):
    if kind == "trees":
        return plain.random_trees(rng, B, T)[0]
    if kind == "one tree":
        return plain.random_trees(rng, 1, T)[0][0]
    if kind == "any":  # not a tree: any nodes, later ones too, and rows that name none
        m = rng.random((B, T, T)) < 0.4
        m[:, ::3] = False
        return m
    return np.zeros((T, T), bool) if kind == "none" else np.ones((B, T, T), bool)


CASES = [
    # B, H, Hk, T, d, page, lengths, mask
    (1, 4, 4, 8, 128, 16, [37], "trees"),
    (1, 1, 1, 1, 64, 8, [1], "trees"),
    (3, 2, 1, 5, 64, 8, [0, 3, 5], "any"),
    (5, 8, 2, 17, 128, 16, [17, 18, 64, 65, 300], "trees"),
    (4, 3, 1, 33, 128, 32, [127, 128, 129, 160], "any"),
    (4, 8, 1, 16, 64, 64, [16, 63, 79, 80], "one tree"),
    (2, 4, 4, 2, 256, 8, [9, 513], "trees"),
    (3, 8, 2, 32, 128, 128, [32, 1500, 3000], "one tree"),
    (2, 16, 4, 64, 256, 32, [64, 900], "trees"),
    (2, 6, 2, 100, 64, 256, [99, 700], "any"),
    (1, 8, 1, 130, 64, 64, [600], "trees"),
    (2, 2, 1, 256, 128, 16, [256, 400], "trees"),
    (1, 3, 1, 256, 256, 8, [300], "any"),
    (2, 4, 2, 7, 128, 16, [7, 200], "none"),
    (2, 4, 2, 7, 128, 16, [6, 200], "all"),
    (70, 2, 2, 3, 64, 16, list(range(70)), "one tree"),
    (1, 40, 1, 8, 64, 16, [333], "trees"),
    (3, 8, 8, 17, 64, 64, [17, 1000, 130], "trees"),
    (3, 8, 1, 4, 64, 8, [200, 4, 131], "any"),
    (2, 4, 2, 31, 64, 32, [900, 129], "any"),
    (2, 1, 1, 64, 64, 16, [64, 192], "trees"),
    (1, 8, 1, 200, 128, 16, [500], "trees"),
    (2, 24, 2, 40, 64, 256, [40, 777], "any"),
    (2, 5, 1, 26, 128, 8, [26, 1300], "any"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])) + "-" + c[7])
def test_matches_the_definition(case):
    import torch

    import flash_attention_gb300 as fa

    B, H, Hk, T, d, ps, lengths, kind = case
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(T + d, B, H, Hk, T, d, ps, lengths)
    m = masks(rng, B, T, kind)
    scale = d ** -0.5
    want = plain.tree_attention(qx, kx, vx, table, lengths, m, scale)
    mask = torch.from_numpy(m).cuda()
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), mask, scale=scale)
    check(got, want)
    # any nonzero byte names a node, and another call gives the same bits
    again = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), mask.byte() * 130,
                                    scale=scale)
    assert all(map(torch.equal, got, again))
    assert fa.fa_device_status(True) == fa.FA_OK


@pytest.mark.parametrize("d,T", [(64, 12), (64, 9), (64, 40), (64, 50), (128, 12), (128, 50), (256, 12)])
def test_long_sequences_of_mixed_lengths(d, T):
    """Sequences that are cut over many CTAs beside some of a few keys."""
    import torch

    import flash_attention_gb300 as fa

    lengths = [9000, 50, 5000, 51, 12345]
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(d, 5, 6, 2, T, d, 32, lengths)
    m = masks(rng, 5, T, "trees")
    want = plain.tree_attention(qx, kx, vx, table, lengths, m, 0.1)
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda(),
                                  scale=0.1)
    check(got, want)


def test_sharp_and_growing_scores():
    """Weights of one key that takes nearly all, and a running maximum that grows along the keys."""
    import torch

    import flash_attention_gb300 as fa

    lengths = [3000, 700]
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(5, 2, 4, 1, 20, 128, 16, lengths)
    for b in range(2):
        j = np.arange(lengths[b])
        kx[table[b][j // 16], 0, j % 16] += qx[b, :, :].mean((0, 1)) * (j / 100)[:, None]
        kx[table[b][j // 16], 0, j % 16, 0] += j / 60
    qx[..., 0] = 4
    (kc, kx), (q, qx) = bf16(kx), bf16(qx)
    m = masks(rng, 2, 20, "trees")
    want = plain.tree_attention(qx, kx, vx, table, lengths, m, 0.125)
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda(),
                                  scale=0.125)
    check(got, want)


def test_a_chain_is_causal_attention():
    import torch

    import flash_attention_gb300 as fa

    lengths = [8, 500, 77]
    _, table, (kc, _), (vc, _), (q, _) = make(1, 3, 8, 2, 8, 128, 16, lengths)
    chain = torch.ones(8, 8, device="cuda").tril().bool()
    o, lse = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), chain, scale=0.1)
    po, pl = fa.paged_attention(q, kc, vc, ints(table), ints(lengths), scale=0.1, causal=True)
    # each within 2^-8 |o| + 2^-8 sum p |v| of the formula (and both alike to 32 bits in L)
    assert (o.float() - po.float()).abs().max() <= 4 * 2 ** -8 * vc.float().abs().max()
    assert (lse - pl).abs().max() <= 2 ** -16 * pl.abs().max()


def test_short_trees_stand_at_the_end():
    """Trees of 3, 5 and 8 nodes in a batch of 8: the same rows as each tree alone gives."""
    import torch

    import flash_attention_gb300 as fa

    sizes, T = [3, 5, 8], 8
    lengths = [3, 50, 200]
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(2, 3, 4, 2, T, 64, 8, lengths)
    m = np.ones((3, T, T), bool)
    alone = []
    for b, n in enumerate(sizes):
        tree = plain.random_trees(rng, 1, n)[0][0]
        m[b, T - n:, T - n:] = tree
        alone.append(plain.tree_attention(qx[b:b + 1, :, T - n:], kx, vx, table[b:b + 1],
                                          lengths[b:b + 1], tree, 0.125))
    o, lse = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths),
                                     torch.from_numpy(m).cuda(), scale=0.125)
    for b, n in enumerate(sizes):
        check((o[b:b + 1, :, T - n:], lse[b:b + 1, :, T - n:]), alone[b])


@pytest.mark.parametrize("d,H", [(64, 2), (64, 4), (64, 6), (64, 12), (128, 6), (128, 12), (256, 6)])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
def test_what_a_node_does_not_see_stays_out(d, what, H):
    """NaN and infinities in the keys and values of some nodes, and everywhere behind the sequences:
    rows that do not see them are as if they were not there; rows that do are what the formula gives."""
    import torch

    import flash_attention_gb300 as fa

    lengths, T = [24, 200, 1000, 131], 24
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(d, 4, H, 2, T, d, 16, lengths)
    m = masks(rng, 4, T, "trees")
    bad = float(what)
    used = np.zeros(kx.shape[:1] + kx.shape[2:3], bool)
    for b, n in enumerate(lengths):
        j = np.arange(n)
        used[table[b][j // 16], j % 16] = True
        for node in (5, 14, 22):
            at = table[b][(n - T + node) // 16], slice(None), (n - T + node) % 16
            if node == 14:
                kx[at] = np.nan  # (an infinite key makes an infinite score or none)
            else:
                vx[at][:, [0, 3, d - 1]] = bad
    for x in (kx, vx):
        x.transpose(0, 2, 1, 3)[~used] = bad
    (kc, kx), (vc, vx) = bf16(kx), bf16(vx)
    with np.errstate(invalid="ignore"):
        want = plain.tree_attention(qx, kx, vx, table, lengths, m, 0.1)
    assert np.isfinite(want[0]).any() and not np.isfinite(want[0]).all()
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda(),
                                  scale=0.1)
    check(got, want)


def test_lengths_and_pages_out_of_range_are_reported():
    import torch

    import flash_attention_gb300 as fa

    lengths = [40, 300]
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(3, 2, 4, 2, 6, 128, 16, lengths)
    P, per = kx.shape[0], table.shape[1]
    m = masks(rng, 2, 6, "trees")
    mask = torch.from_numpy(m).cuda()
    for bad_len, entry in (([-5, 300], None), ([per * 16 + 1, 300], None), (lengths, P),
                           (lengths, -1), (lengths, 2 ** 31 - 1)):
        t = table.copy()
        if entry is not None:
            t[1, 3] = t[0, 2] = entry
        want = plain.tree_attention(qx, kx, vx, t, np.array(bad_len), m, 0.1)
        got = fa.paged_tree_attention(q, kc, vc, ints(t), ints(bad_len), mask, scale=0.1)
        assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT, (bad_len, entry)
        check(got, want)
    # entries that no key is in are not looked at
    t = table.copy()
    t[0, 3:] = -7
    got = fa.paged_tree_attention(q, kc, vc, ints(t), ints(lengths), mask, scale=0.1)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_shared_prefix_pages():
    """Sequences whose tables name the same pages (a shared prefix is only read)."""
    import torch

    import flash_attention_gb300 as fa

    lengths = [70, 90, 80]
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(4, 3, 2, 1, 9, 64, 16, lengths)
    table[:, :3] = table[0, :3]
    m = masks(rng, 3, 9, "trees")
    want = plain.tree_attention(qx, kx, vx, table, lengths, m, 0.2)
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda(),
                                  scale=0.2)
    check(got, want)


def test_a_cache_past_32_bits():
    import torch

    import flash_attention_gb300 as fa

    Hk, ps, d, T = 8, 256, 128, 10
    P = (1 << 31) // (Hk * ps * d) + 40
    kc = torch.zeros(P, Hk, ps, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rng = np.random.default_rng(1)
    table = np.array([[P - 1, 2, P - 30, P - 7]])
    x = [bf16(rng.standard_normal((4, Hk, ps, d))) for _ in range(2)]
    kc[table[0].tolist()], vc[table[0].tolist()] = x[0][0], x[1][0]
    q, qx = bf16(rng.standard_normal((1, 16, T, d)))
    m = masks(rng, 1, T, "trees")
    want = plain.tree_attention(qx, x[0][1], x[1][1], np.arange(4)[None], [1000], m, 0.1)
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints([1000]), torch.from_numpy(m).cuda(),
                                  scale=0.1)
    check(got, want)


def test_graphs_replayed_at_once():
    """Graphs of several calls each, replayed on streams of their own while the current stream runs
    the same calls: each has scratch of its own."""
    import torch

    import flash_attention_gb300 as fa

    lengths = [3000, 700, 20, 250]
    rng, table, (kc, _), (vc, _), _ = make(6, 4, 8, 2, 20, 128, 16, lengths)
    tb, lens = ints(table), ints(lengths)
    work = [(bf16(rng.standard_normal((4, 8, T, 128)))[0],
             torch.from_numpy(masks(rng, 4, T, "trees")).cuda()) for T in (1, 4, 20, 64)]

    def calls(q, m):
        return [fa.paged_tree_attention(q, kc, vc, tb, lens, m, scale=0.1) for _ in range(4)]

    want = [calls(*x)[0] for x in work]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for x in work:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(calls(*x))
    streams = [torch.cuda.Stream() for _ in work]
    for i in range(10):
        for x in outs:
            for o, lse in x:
                o.fill_(7)
                lse.fill_(7)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = calls(*work[i % 4])
        torch.cuda.synchronize()
        for x, (o, lse) in zip([*outs, eager], [*want, want[i % 4]]):
            assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in x)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_outputs_stay_within_their_bounds():
    """o and lse inside larger buffers: what lies around them is left as it was, all of them written."""
    import ctypes

    import torch

    import flash_attention_gb300 as fa

    for (B, H, Hk, T, d, ps, lengths, kind) in CASES[2:9]:
        rng, table, (kc, _), (vc, _), (q, _) = make(T, B, H, Hk, T, d, ps, lengths)
        m = torch.from_numpy(np.broadcast_to(masks(rng, B, T, kind), (B, T, T)).copy()).cuda()
        tb, lens = ints(table), ints(lengths)
        o = torch.full((q.numel() + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B * H * T + 64,), 7.0, device="cuda")
        p = fa.FaPagedParams(B, H, Hk, T, d, ps, table.shape[1], kc.shape[0], 0.1, 0, 0, 0)
        rc = fa.load_library().fa_paged_tree_attention(
            q.data_ptr(), kc.data_ptr(), vc.data_ptr(), tb.data_ptr(), lens.data_ptr(),
            m.data_ptr(), T * T, o[128:].data_ptr(), lse[32:].data_ptr(), ctypes.byref(p),
            torch.cuda.current_stream().cuda_stream)
        assert rc == fa.FA_OK
        want = fa.paged_tree_attention(q, kc, vc, tb, lens, m, scale=0.1)
        assert torch.equal(o[128:-128].view_as(q), want[0])
        assert torch.equal(lse[32:-32].view(B, H, T), want[1])
        assert (o[:128] == 7).all() and (o[-128:] == 7).all()
        assert (lse[:32] == 7).all() and (lse[-32:] == 7).all()


def test_on_another_stream():
    import torch

    import flash_attention_gb300 as fa

    lengths = [500, 40]
    rng, table, (kc, _), (vc, _), (q, _) = make(8, 2, 4, 2, 9, 128, 16, lengths)
    m = torch.from_numpy(masks(rng, 2, 9, "trees")).cuda()
    args = q, kc, vc, ints(table), ints(lengths), m
    want = fa.paged_tree_attention(*args, scale=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.paged_tree_attention(*args, scale=0.1, stream=s)
    s.synchronize()
    assert all(map(torch.equal, got, want))


@pytest.mark.parametrize("d,T", [(64, 9), (64, 30), (64, 60), (64, 80), (128, 9), (128, 80),
                                 (256, 9)])
def test_waits_that_run_out_are_reported(d, T):
    """With a limit of 1 ns the kernel's ordinary waits run out: it winds down, the status says so, and
    with the limit restored the same call is right."""
    import torch

    import flash_attention_gb300 as fa

    lengths = [3000, 700]
    rng, table, (kc, kx), (vc, vx), (q, qx) = make(d, 2, 4, 2, T, d, 16, lengths)
    m = masks(rng, 2, T, "trees")
    args = q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda()
    try:
        fa.fa_set_wait_limit_ns(1)
        fa.paged_tree_attention(*args, scale=0.1)
        assert fa.fa_device_status(True) == fa.FA_ERR_DEVICE_TIMEOUT
    finally:
        fa.fa_set_wait_limit_ns(0)
    got = fa.paged_tree_attention(*args, scale=0.1)
    assert fa.fa_device_status(True) == fa.FA_OK
    check(got, plain.tree_attention(qx, kx, vx, table, lengths, m, 0.1))


def test_a_batch_of_thousands():
    """More sequences than any warp looks at at once, most of them empty or of a few keys."""
    import torch

    import flash_attention_gb300 as fa

    B, T = 3000, 3
    rng = np.random.default_rng(12)
    lengths = np.where(rng.random(B) < 0.5, 0, rng.integers(1, 20, B))
    lengths[[7, 1500, B - 1]] = [700, 300, 64]
    per = 44
    table = np.zeros((B, per), np.int32)
    used = -(-lengths // 16)
    pages = rng.permutation(int(used.sum()) + 2)
    at = 0
    for b in range(B):
        table[b, :used[b]] = pages[at:at + used[b]]
        at += used[b]
    P = len(pages)
    (kc, kx), (vc, vx) = (bf16(rng.standard_normal((P, 1, 16, 64))) for _ in range(2))
    q, qx = bf16(rng.standard_normal((B, 2, T, 64)))
    m = masks(rng, B, T, "one tree")
    want = plain.tree_attention(qx, kx, vx, table, lengths, m, 0.125)
    got = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(m).cuda(),
                                  scale=0.125)
    check(got, want)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_masks_of_any_batch_stride_and_alignment():
    import torch

    import flash_attention_gb300 as fa

    for T in (7, 8, 33, 64):
        lengths = [300, 70, 200]
        rng, table, (kc, kx), (vc, vx), (q, qx) = make(T, 3, 2, 1, T, 128, 16, lengths)
        m = masks(rng, 3, T, "any")
        want = plain.tree_attention(qx, kx, vx, table, lengths, m, 0.1)
        for stride, off in ((T * T, 0), (T * T + 3, 1), (2 * T * T, 2)):
            flat = torch.ones(4 * stride + 8, dtype=torch.uint8, device="cuda")
            view = flat.as_strided((3, T, T), (stride, T, 1), off)
            view.copy_(torch.from_numpy(m).cuda())
            check(fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), view, scale=0.1), want)


def test_a_captured_call_takes_the_lengths_of_its_replay():
    import torch

    import flash_attention_gb300 as fa

    rng, table, (kc, kx), (vc, vx), (q, qx) = make(9, 3, 8, 2, 12, 128, 16, [2000, 2000, 2000])
    m = masks(rng, 3, 12, "trees")
    lens, mask, tb = ints([100, 2000, 0]), torch.from_numpy(m).cuda(), ints(table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.paged_tree_attention(q, kc, vc, tb, lens, mask, scale=0.1)
    for lengths in ([100, 2000, 0], [12, 13, 14], [0, 0, 0], [2000, 5, 1999]):
        lens.copy_(ints(lengths))
        graph.replay()
        check(got, plain.tree_attention(qx, kx, vx, table, lengths, m, 0.1))
    assert fa.fa_device_status(True) == fa.FA_OK
