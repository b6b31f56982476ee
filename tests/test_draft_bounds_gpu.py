"""Drafted decoding held to bounds that a wrong value of one drafted node would pass: each element of a
chain against causal attention, and the answers of whole steps against the plain form on the queries and
keys that the cache holds.

Each kernel's O is within 2^-8 |o| + (2^-8 + 2^-14) sum p |v| of the formula (tests/test_tree_gpu.py), so two
kernels are within twice that of one another, |o| being either's to a rounding of the same size."""
import numpy as np
import pytest

from tests import draft_plain as plain
from tests.test_rotary_gpu import _gpu, bf16, freqs, ints  # noqa: F401
from tests.test_tree_gpu import check, make

pytestmark = pytest.mark.gpu


def apart(a, b, want):
    """Largest error of o in units of the bound for two kernels, and that of L."""
    a, b = ([t.double().cpu().numpy() for t in x] for x in (a, b))
    o, lse, w = want
    bound = 2 * (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -14) * w) + 1e-30
    return (np.abs(a[0] - b[0]) / bound).max(), np.abs(a[1] - b[1]).max() / np.abs(lse).max()


@pytest.mark.parametrize("case", [(8, 2, 8, 128, 16), (4, 4, 17, 64, 64), (8, 1, 5, 256, 8), (6, 2, 1, 64, 32)],
                         ids=str)
def test_a_chain_is_causal_attention(case):
    import torch

    import flash_attention_gb300 as fa

    H, Hk, T, d, ps = case
    lengths = [T, 500, 77]
    _, table, (kc, kx), (vc, vx), (q, qx) = make(T, 3, H, Hk, T, d, ps, lengths)
    tril = np.tril(np.ones((T, T), bool))
    want = plain.tree_attention(qx, kx, vx, table, lengths, tril, 0.1)
    tree = fa.paged_tree_attention(q, kc, vc, ints(table), ints(lengths), torch.from_numpy(tril).cuda(),
                                   scale=0.1)
    chain = fa.paged_attention(q, kc, vc, ints(table), ints(lengths), scale=0.1, causal=True)
    check(tree, want)
    o, lse = apart(tree, chain, want)
    assert o <= 1 and lse <= 2 ** -16
    # the bound tells: without the drafted nodes' values it is passed
    vx[table[1][np.arange(500 - T, 500) // ps], :, np.arange(500 - T, 500) % ps] = 0
    o = plain.tree_attention(qx, kx, vx, table, lengths, tril, 0.1)[0]
    bound = 2 * (2.0 ** -8 * np.abs(want[0]) + (2.0 ** -8 + 2.0 ** -14) * want[2])
    assert (np.abs(o - want[0])[1] > bound[1]).any()


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("shape", [(4, 2, 128, 16, 11), (8, 8, 64, 64, 20), (4, 1, 256, 8, 6)], ids=str)
def test_steps_on_what_the_cache_holds(shape, inter):
    """Append, attend, keep, three times; every step's answers against the plain form on the returned
    queries and the cache as they are read back, and the next token's by the cache's other reader."""
    import torch

    import flash_attention_gb300 as fa

    H, Hk, d, ps, T = shape
    rng = np.random.default_rng(T + 100)
    prompts, rot, scale = [37, 1, 150], d // 2, d ** -0.5
    B = len(prompts)
    table, P = plain.make_table(rng, B, (max(prompts) + 4 * T) // ps + 2)
    tb, f = ints(table), freqs(plain.inv_freq(rot))
    kc, vc = (torch.zeros(P, Hk, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    total, cu = sum(prompts), np.concatenate([[0], np.cumsum(prompts)])
    k, v = (bf16(rng.standard_normal((Hk, total, d)))[0] for _ in range(2))
    lengths = ints(prompts)
    fa.paged_cache_append(k, v, kc, vc, tb, lengths, inv_freq=f, interleaved=inter, cu_seqlens=ints(cu))
    for step in range(3):
        sees, _ = plain.random_trees(rng, B, T, most=3)
        depth = sees.sum(-1) - 1
        q, k, v = (bf16(rng.standard_normal((B, n, T, d)))[0] for n in (H, Hk, Hk))
        pos = lengths.cpu().numpy()[:, None] + depth
        lengths = lengths + T
        qt = fa.paged_cache_append(k, v, kc, vc, tb, lengths, q=q, inv_freq=f, interleaved=inter,
                                   positions=ints(pos))
        got = fa.paged_tree_attention(qt, kc, vc, tb, lengths, torch.from_numpy(sees).cuda(), scale=scale)
        qx, kx, vx = (t.double().cpu().numpy() for t in (qt, kc, vc))
        at = lengths.cpu().numpy()
        check(got, plain.tree_attention(qx, kx, vx, table, at, sees, scale))
        for b in range(B):  # what was appended is the rows' values, and their keys turned
            for x, cache, turned in ((k, kx, True), (v, vx, False)):
                rows = x[b].double().cpu().numpy()
                want = plain.turn(rows, pos[b], plain.inv_freq(rot), inter) if turned else rows
                bound = plain.turn_bound(rows, want, rot, inter, 1.0) if turned else 0
                have = plain.keys_of(cache, table[b], at[b])[:, at[b] - T:]
                assert (np.abs(have - want) <= bound).all()
        leaf = rng.integers(0, T, B)
        paths = [np.flatnonzero(sees[b, leaf[b]]) for b in range(B)]
        keep = np.zeros((B, max(map(len, paths))), int)
        for b in range(B):
            keep[b, :len(paths[b])] = paths[b]
        lengths = fa.paged_cache_keep(kc, vc, tb, lengths, ints(keep), ints([len(x) for x in paths]), T)
    q, qx = bf16(rng.standard_normal((B, H, 1, d)))
    one = torch.ones(1, 1, dtype=torch.bool, device="cuda")
    want = plain.tree_attention(qx, kc.double().cpu().numpy(), vc.double().cpu().numpy(), table,
                                lengths.cpu().numpy(), np.ones((1, 1), bool), scale)
    tree = fa.paged_tree_attention(q, kc, vc, tb, lengths, one, scale=scale)
    check(tree, want)
    o, lse = apart(tree, fa.paged_attention(q, kc, vc, tb, lengths, scale=scale), want)
    assert o <= 1 and lse <= 2 ** -15
    assert fa.fa_device_status(True) == fa.FA_OK
