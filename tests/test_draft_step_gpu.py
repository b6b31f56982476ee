"""Drafted decoding as a program runs it: prompts appended with their rotation, then step after step a
tree appended, attended and cut back to an accepted path; at the end the cache has to be that of the
accepted tokens alone, and every step's attention that of each node's path."""
import numpy as np
import pytest

from tests import draft_plain as plain
from tests.test_rotary_gpu import _gpu, bf16, freqs, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("shape", [(4, 2, 128, 16, 11), (8, 8, 64, 64, 20), (4, 1, 256, 8, 6)], ids=str)
def test_steps(shape, inter):
    import torch

    import flash_attention_gb300 as fa

    H, Hk, d, ps, T = shape
    rng = np.random.default_rng(T)
    prompts, rot, scale = [37, 1, 150], d // 2, d ** -0.5
    B = len(prompts)
    table, P = plain.make_table(rng, B, (max(prompts) + 5 * T) // ps + 2)
    tb, f = ints(table), freqs(plain.inv_freq(rot))
    kc, vc = (torch.full((P, Hk, ps, d), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    total = sum(prompts)
    cu = np.concatenate([[0], np.cumsum(prompts)])
    wide, wx = bf16(rng.standard_normal((total, H + 2 * Hk, d)))  # one projection's output
    heads = wide.transpose(0, 1)
    lengths = ints(prompts)
    fa.paged_cache_append(heads[H:H + Hk], heads[H + Hk:], kc, vc, tb, lengths, q=heads[:H],
                          inv_freq=f, interleaved=inter, cu_seqlens=ints(cu))
    path = [[(wx[i, H:H + Hk], wx[i, H + Hk:]) for i in range(cu[b], cu[b + 1])] for b in range(B)]

    def turned(rows):  # [Hk, n, d] of a path's (k, v), the keys at their positions
        k = np.stack([r[0] for r in rows], 1)
        return plain.turn(k, np.arange(len(rows)), plain.inv_freq(rot), inter)

    for step in range(4):
        sees, parents = plain.random_trees(rng, B, T, most=3)
        depth = sees.sum(-1) - 1
        new, nx = bf16(rng.standard_normal((B, T, H + 2 * Hk, d)))
        q, k, v = new.transpose(1, 2).split((H, Hk, Hk), 1)
        before = np.array([len(p) for p in path])
        lengths = lengths + T
        qt = fa.paged_cache_append(k, v, kc, vc, tb, lengths, q=q, inv_freq=f, interleaved=inter,
                                   positions=ints(before[:, None] + depth))
        o, lse = fa.paged_tree_attention(qt, kc, vc, tb, lengths, torch.from_numpy(sees).cuda(),
                                         scale=scale)
        o, kept = o.double().cpu().numpy(), []
        for b in range(B):
            for node in range(T):  # a node's answer is that of its path alone
                rows = path[b] + [(nx[b, i, H:H + Hk], nx[b, i, H + Hk:])
                                  for i in np.flatnonzero(sees[b, node])]
                kk, vv = turned(rows), np.stack([r[1] for r in rows], 1)
                qq = plain.turn(nx[b, node, :H][:, None], np.array([before[b] + depth[b, node]]),
                                plain.inv_freq(rot), inter)[:, 0]
                for h in range(H):
                    s = kk[h // (H // Hk)] @ qq[h] * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    vh = vv[h // (H // Hk)]
                    # q and k are rounded once more here (2^-8 of each element): a score is off by
                    # ds = 2 * 2^-8 sum |q k| scale at most, a weight by a factor of e^(2 ds), beside
                    # what tests/test_tree_gpu.py counts
                    ds = 2.0 ** -7 * (np.abs(kk[h // (H // Hk)]) @ np.abs(qq[h])).max() * scale
                    bound = 2.0 ** -8 * np.abs(p @ vh) + (np.expm1(2 * ds) + 2.0 ** -7) * (p @ np.abs(vh))
                    assert (np.abs(o[b, h, node] - p @ vh) <= bound).all()
            leaf = int(rng.integers(0, T))
            kept.append(np.flatnonzero(sees[b, leaf]) if step != 2 or b else np.zeros(0, int))
        M = max(1, max(len(x) for x in kept))
        keep = np.zeros((B, M), int)
        for b in range(B):
            keep[b, :len(kept[b])] = kept[b]
            path[b] += [(nx[b, i, H:H + Hk], nx[b, i, H + Hk:]) for i in kept[b]]
        lengths = fa.paged_cache_keep(kc, vc, tb, lengths, ints(keep), ints([len(x) for x in kept]),
                                      T)
        assert lengths.tolist() == [len(p) for p in path]
    kx, vx = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    for b in range(B):
        n = len(path[b])
        want = turned(path[b])
        x = np.stack([r[0] for r in path[b]], 1)
        err = np.abs(plain.keys_of(kx, table[b], n) - want)
        assert (err <= plain.turn_bound(x, want, rot, inter, 1.0)).all()
        np.testing.assert_array_equal(plain.keys_of(vx, table[b], n),
                                      np.stack([r[1] for r in path[b]], 1))
    # and the next token of the accepted text, by the cache's other reader
    q, _ = bf16(rng.standard_normal((B, H, 1, d)))
    one = torch.ones(1, 1, dtype=torch.bool, device="cuda")
    a = fa.paged_tree_attention(q, kc, vc, tb, lengths, one, scale=scale)
    c = fa.paged_attention(q, kc, vc, tb, lengths, scale=scale)
    assert (a[0].float() - c[0].float()).abs().max() <= 2 ** -6 * vc[vc.isfinite()].abs().max()
    assert (a[1] - c[1]).abs().max() <= 2 ** -15 * max(1.0, float(c[1].abs().max()))
    assert fa.fa_device_status(True) == fa.FA_OK
