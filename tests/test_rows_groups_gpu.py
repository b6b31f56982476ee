"""Rotation and appending where the rows alone fill the GPU, so that a CTA walks over 8 heads, with
counts of heads that are no multiple of 8 or of the 4 whose loads are in flight; and kept rows wider
than one block's columns."""
import numpy as np
import pytest

from tests import draft_plain as plain, test_paged_append_gpu as rows
from tests.test_rotary_gpu import _gpu, bf16, check, freqs, ints, laid_out  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("case", [(2, 9, 3, 4000, 64, 32, "fused"), (1, 21, 5, 2600, 128, 128, "rows"),
                                  (3, 13, 2, 900, 256, 64, "heads")], ids=str)
def test_rotation(case, back):
    import flash_attention_gb300 as fa

    B, H, Hk, n, d, rot, layout = case
    rng = np.random.default_rng(n)
    q, qx = laid_out(rng.standard_normal((B, H, n, d)), layout)
    k, kx = laid_out(rng.standard_normal((B, Hk, n, d)), layout)
    freq = plain.inv_freq(rot)
    call = fa.rotary_bwd if back else fa.rotary_fwd
    for inter in (False, True):
        qo, ko = call(q, k, freqs(freq), interleaved=inter, scale=1.25, offset=3)
        check(qo, qx, np.arange(n) + 3, freq, inter, 1.25, back)
        check(ko, kx, np.arange(n) + 3, freq, inter, 1.25, back)
    if layout != "heads":  # in place
        fa_q, fa_k = q.clone(), k.clone()
        call(fa_q, fa_k, freqs(freq), interleaved=True, scale=1.25, offset=3, out=(fa_q, fa_k))
        assert (fa_q == qo).all() and (fa_k == ko).all()


@pytest.mark.parametrize("case", [(13, 9, 64, 32, 16), (9, 3, 128, 128, 8), (5, 10, 256, 96, 64)], ids=str)
def test_appending(case):
    """Prompts of mixed lengths with their queries."""
    import flash_attention_gb300 as fa

    H, Hk, d, rot, ps = case
    rng = np.random.default_rng(d)
    past, new = np.array([0, 5, 300, 17]), np.array([1500, 2000, 1, 2300])
    lengths, B, total = past + new, 4, int(new.sum())
    cu = np.concatenate([[0], np.cumsum(new)])
    table, P = plain.make_table(rng, B, int(-(-lengths.max() // ps)))
    (kc, kcx), (vc, vcx) = (bf16(rng.standard_normal((P, Hk, ps, d))) for _ in range(2))
    q, qx = laid_out(rng.standard_normal((H, total, d)), "fused")
    k, kx = laid_out(rng.standard_normal((Hk, total, d)), "fused")
    v, vx = laid_out(rng.standard_normal((Hk, total, d)), "rows")
    freq = plain.inv_freq(rot)
    qo = fa.paged_cache_append(k, v, kc, vc, ints(table), ints(lengths), q=q, inv_freq=freqs(freq),
                               cu_seqlens=ints(cu))
    pos = np.concatenate([np.arange(m - n, m) for m, n in zip(lengths, new)])
    check(qo, qx, pos, freq, False, 1.0, False)
    turned = plain.turn(kx, pos, freq)
    slack = plain.turn_bound(kx, turned, rot, False, 1.0)
    slack[..., rot:] = 0
    cut = [slice(cu[b], cu[b + 1]) for b in range(B)]
    bound = np.zeros_like(kcx)
    plain.append(kcx, vcx, [turned[:, s] for s in cut], [vx[:, s] for s in cut], table, lengths)
    plain.append(bound, bound.copy(), *([slack[:, s] for s in cut],) * 2, table, lengths)
    assert (np.abs(kc.double().cpu().numpy() - kcx) <= bound).all()
    np.testing.assert_array_equal(vc.double().cpu().numpy(), vcx)
    assert fa.fa_device_status(True) == fa.FA_OK


@pytest.mark.parametrize("case", [(16, 128, 16, 12, 7, [12, 40, 33]), (9, 256, 8, 20, 20, [20, 57]),
                                  (40, 64, 32, 5, 3, [5, 64, 100])], ids=str)
def test_keeping(case):
    rows.test_keep_moves_the_accepted_rows(case)


def test_no_rows_and_no_heads():
    """Nothing to turn gives empty outputs; keys without queries are refused, not left unturned."""
    import torch

    import flash_attention_gb300 as fa

    f, _ = fa.rotary_inv_freq(64)
    x = torch.ones(2, 4, 6, 64, dtype=torch.bfloat16, device="cuda")
    for q, k in ((x[:, :, :0], x[:, :2, :0]), (x[:0], x[:0, :2]), (x[0, :, :0], None)):
        qo, ko = fa.rotary_fwd(q, k, f)
        assert qo.shape == q.shape and (k is None or ko.shape == k.shape)
    for q, k in ((x[:, :0], x), (x[0, :0], x[0]), (x[:, :0], None)):
        with pytest.raises(fa.FaError):
            fa.rotary_fwd(q, k, f)
