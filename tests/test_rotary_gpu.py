"""Rotary positions on the GPU against the plain 64-bit form, element by element (the bound is
tests.draft_plain.turn_bound's), and their gradient."""
import numpy as np
import pytest

from tests import draft_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import flash_attention_gb300 as fa

    fa.build()
    fa.fa_device_status(True)
    yield
    fa.fa_device_status(True)


def bf16(x):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().cuda()
    return t, t.double().cpu().numpy()


def ints(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def freqs(f):
    import torch

    return torch.from_numpy(np.ascontiguousarray(f, np.float64)).cuda()


def laid_out(x, layout):
    """A bf16 tensor [.., heads, rows, d] of the values x, in memory as `layout` says."""
    import torch

    t, x = bf16(x)
    if layout == "rows":
        t = t.transpose(-3, -2).contiguous().transpose(-3, -2)
    elif layout == "fused":  # columns of a wider projection
        H, n, d = t.shape[-3:]
        wide = torch.full((*t.shape[:-3], n, H + 3, d), float("nan"), dtype=t.dtype, device="cuda")
        wide[..., 2:2 + H, :] = t.transpose(-3, -2)
        t = wide[..., 2:2 + H, :].transpose(-3, -2)
    return t, x


def check(got, x, pos, freq, inter, scale, back):
    want = plain.turn(x, pos, freq, inter, scale, back)
    err = np.abs(got.double().cpu().numpy() - want)
    bound = plain.turn_bound(x, want, 2 * len(freq), inter, scale)
    assert (err <= bound).all(), (err / bound).max()
    rot = 2 * len(freq)
    np.testing.assert_array_equal(got.double().cpu().numpy()[..., rot:], x[..., rot:])


CASES = [  # B, H, Hk, n, d, rot
    (1, 1, 1, 1, 64, 64), (2, 4, 2, 7, 128, 128), (3, 3, 1, 65, 64, 16), (1, 8, 8, 33, 256, 256),
    (2, 5, 5, 100, 128, 96), (1, 2, 1, 9, 256, 48), (2, 9, 3, 130, 64, 32), (5, 16, 2, 3, 128, 32),
    (1, 70, 1, 2, 64, 48),
]


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("layout", ["heads", "rows", "fused"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_matches_the_definition(case, layout, inter, back):
    import flash_attention_gb300 as fa

    B, H, Hk, n, d, rot = case
    rng = np.random.default_rng(B * 1000 + n + rot)
    q, qx = laid_out(rng.standard_normal((B, H, n, d)), layout)
    k, kx = laid_out(rng.standard_normal((B, Hk, n, d)) * 3, layout)
    freq = plain.inv_freq(rot)
    call = fa.rotary_bwd if back else fa.rotary_fwd
    scale = 1.0 if n % 2 else 0.75
    qo, ko = call(q, k, freqs(freq), interleaved=inter, scale=scale, offset=11)
    pos = np.arange(n) + 11
    check(qo, qx, pos, freq, inter, scale, back)
    check(ko, kx, pos, freq, inter, scale, back)
    assert qo.is_contiguous() or qo.transpose(1, 2).is_contiguous()
    own = rng.integers(-50, 200000, (B, n))  # positions of their own for each sequence, or for all
    qo, ko = call(q, k, freqs(freq), interleaved=inter, scale=scale, positions=ints(own))
    check(qo, qx, own[:, None], freq, inter, scale, back)
    check(ko, kx, own[:, None], freq, inter, scale, back)
    qo, none = call(q, None, freqs(freq), interleaved=inter, scale=scale, positions=ints(own[0]))
    check(qo, qx, own[0], freq, inter, scale, back)
    assert none is None
    assert fa.fa_device_status(True) == fa.FA_OK


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("lens", [[5], [1, 0, 0, 130, 7], [0, 3, 64, 0], [1] * 70])
def test_packed_sequences_count_from_their_first_row(lens, inter):
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(len(lens))
    total, d, rot = sum(lens), 128, 64
    rows = total + 3  # the last three belong to no sequence
    q, qx = laid_out(rng.standard_normal((4, rows, d)), "rows")
    k, kx = laid_out(rng.standard_normal((2, rows, d)), "heads")
    freq = plain.inv_freq(rot)
    cu = ints(np.concatenate([[0], np.cumsum(lens)]))
    out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    qo, ko = fa.rotary_fwd(q, k, freqs(freq), cu_seqlens=cu, offset=1000, interleaved=inter, out=out)
    pos = np.concatenate([np.arange(n) for n in lens]) + 1000
    check(qo[:, :total], qx[:, :total], pos, freq, inter, 1.0, False)
    check(ko[:, :total], kx[:, :total], pos, freq, inter, 1.0, False)
    assert (qo[:, total:] == 7).all() and (ko[:, total:] == 7).all()
    # positions given for every packed row, and none at all: one sequence
    own = rng.integers(0, 1 << 20, rows)
    qo, ko = fa.rotary_fwd(q, k, freqs(freq), positions=ints(own), interleaved=inter)
    check(qo, qx, own, freq, inter, 1.0, False)
    qo, ko = fa.rotary_fwd(q, k, freqs(freq), interleaved=inter)
    check(ko, kx, np.arange(rows), freq, inter, 1.0, False)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_far_positions_and_any_frequencies():
    """The angle is right at the first and the last 32-bit positions, for frequencies above a turn a
    position, negative ones, 0 and subnormal numbers."""
    import flash_attention_gb300 as fa

    pos = np.array([-2 ** 31, -2 ** 31 + 1, -1, 0, 1, 999999, 2 ** 24 + 1, 2 ** 31 - 1])
    freq = np.array([1.0, 0.5, 1e-5, 6.25, -1.0, 0.0, 5e-324, 1e-300, 3.9, 2.0 ** -31, 1 / 3, 0.1,
                     -7e-3, 1e-9, 2 * np.pi, 1.9999])
    rng = np.random.default_rng(3)
    q, qx = bf16(rng.standard_normal((1, 2, 8, 64)))
    qo, _ = fa.rotary_fwd(q, None, freqs(freq), positions=ints(pos))
    # (frequencies up to 8: 2^3 times 2^-30 of a turn at most, below 2^-24)
    check(qo, qx, pos, freq, False, 1.0, False)


def test_values_that_are_not_finite_stay_in_their_pair():
    import flash_attention_gb300 as fa

    rng = np.random.default_rng(4)
    x = rng.standard_normal((1, 1, 5, 128))
    x[0, 0, 1, 3], x[0, 0, 2, 40], x[0, 0, 3, 100], x[0, 0, 3, 127] = np.nan, np.inf, np.nan, -np.inf
    q, qx = bf16(x)
    freq = plain.inv_freq(64)
    freq[5] = np.nan
    for inter in (False, True):
        got = fa.rotary_fwd(q, None, freqs(freq), interleaved=inter)[0].double().cpu().numpy()
        want = plain.turn(qx, np.arange(5), freq, inter)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        np.testing.assert_array_equal(got[..., 64:], qx[..., 64:])
        inf = np.isinf(want)
        np.testing.assert_array_equal(got[inf], want[inf])


def test_in_place_and_back_again():
    import torch

    import flash_attention_gb300 as fa

    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, 50, 8, 128, generator=g, device="cuda").bfloat16().transpose(1, 2)
    k = torch.randn(2, 2, 50, 128, generator=g, device="cuda").bfloat16()
    f, scale = fa.rotary_inv_freq(128)
    assert scale == 1.0
    want = fa.rotary_fwd(q, k, f)
    assert want[0].stride() == q.stride() and want[1].is_contiguous()
    q2, k2 = q.clone(), k.clone()
    assert q2.stride() == q.stride()
    got = fa.rotary_fwd(q2, k2, f, out=(q2, k2))
    assert got[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    fa.rotary_bwd(q2, k2, f, out=(q2, k2))
    # two roundings of 2^-8, and the turn keeps a pair's length
    assert (q2.float() - q.float()).abs().max() <= 2 ** -6.5 * q.float().abs().max()


def test_gradient_of_attention_on_turned_rows():
    """d loss / d q of <dO, attention(rotary(q), rotary(k), v)> against central differences in 64 bits
    of the formula, and against its closed form, on a tiny problem. What the kernels compute in bf16
    is q' and k' (each within turn_bound), O, dq', dk' and the turned-back gradients; their errors come
    to a few 2^-8 of the largest gradient, and 2e-2 of it is the bound that attention's own gradients
    are held to."""
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(8)
    B, H, Hk, n, d, rot = 1, 2, 1, 6, 64, 32
    freq, scale = plain.inv_freq(rot), d ** -0.5
    q, qx = bf16(rng.standard_normal((B, H, n, d)))
    k, kx = bf16(rng.standard_normal((B, Hk, n, d)))
    v, vx = bf16(rng.standard_normal((B, Hk, n, d)))
    do, dox = bf16(rng.standard_normal((B, H, n, d)))
    f = freqs(freq)
    qt, kt = fa.rotary_fwd(q, k, f, interleaved=True)
    o, lse = fa.attention_fwd(qt, kt, v, scale=scale, causal=True)
    dqt, dkt, _ = fa.attention_bwd(qt, kt, v, o, lse, do, scale=scale, causal=True)
    dq, dk = fa.rotary_bwd(dqt, dkt, f, interleaved=True)

    def loss(qx, kx):
        a, b = (plain.turn(x, np.arange(n), freq, True) for x in (qx, kx))
        s = np.einsum("bhid,bjd->bhij", a, b[:, 0]) * scale
        s = np.where(np.tril(np.ones((n, n), bool)), s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        return np.sum(np.einsum("bhij,bjd->bhid", p, vx[:, 0]) * dox)

    for got, at in ((dq, 0), (dk, 1)):
        got = got.double().cpu().numpy()
        want = np.zeros_like(got)
        for i in np.ndindex(*got.shape):
            xs = [qx.copy(), kx.copy()], [qx.copy(), kx.copy()]
            xs[0][at][i] += 1e-5
            xs[1][at][i] -= 1e-5
            want[i] = (loss(*xs[0]) - loss(*xs[1])) / 2e-5
        assert np.abs(got - want).max() <= 2e-2 * np.abs(want).max()


def test_the_gradient_is_the_transpose():
    """<rotary(x), y> = <x, rotary_bwd(y)>: the backward pass against the formula's gradient."""
    import flash_attention_gb300 as fa

    rng = np.random.default_rng(9)
    freq = plain.inv_freq(64)
    for inter in (False, True):
        y, yx = bf16(rng.standard_normal((1, 3, 20, 128)))
        got = fa.rotary_bwd(y, None, freqs(freq), interleaved=inter, scale=1.25)[0]
        eye = np.eye(128)  # the Jacobian's columns, at each position
        for p in range(20):
            J = plain.turn(eye, np.full(128, p), freq, inter, 1.25).T  # y = J x
            want = yx[:, :, p] @ J
            err = np.abs(got[:, :, p].double().cpu().numpy() - want)
            assert (err <= plain.turn_bound(yx[:, :, p], want, 64, inter, 1.25) + 1e-12).all()


def test_captured_and_on_another_stream():
    import torch

    import flash_attention_gb300 as fa

    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(3, 8, 129, 64, generator=g, device="cuda").bfloat16()
    k = torch.randn(3, 2, 129, 64, generator=g, device="cuda").bfloat16()
    f, _ = fa.rotary_inv_freq(64)
    want = fa.rotary_fwd(q, k, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.rotary_fwd(q, k, f, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.rotary_fwd(q, k, f)
        back = fa.rotary_bwd(*got, f)
    x = torch.randn_like(q)
    q.copy_(x)
    graph.replay()
    want = fa.rotary_fwd(q, k, f)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(back, fa.rotary_bwd(*want, f)))


def test_offsets_out_of_range_are_reported():
    import torch

    import flash_attention_gb300 as fa

    q = torch.ones(1, 10, 64, dtype=torch.bfloat16, device="cuda")
    f, _ = fa.rotary_inv_freq(64)
    for cu in ([0, 11], [0, 5, 3, 10], [1, 10], [-1, 10], [0, 2 ** 31 - 1]):
        out = torch.full_like(q, 7.0)
        fa.rotary_fwd(q, None, f, cu_seqlens=ints(cu), out=(out, None))
        assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT, cu
    assert fa.fa_device_status(True) == fa.FA_OK


def test_rows_past_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements: the rows of its last head."""
    import torch

    import flash_attention_gb300 as fa

    H, n, d = 40, 1 << 19, 128
    q = torch.zeros(1, H, n, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(2, 64, d, device="cuda").bfloat16()
    q[0, -2:, -64:] = tail
    f, _ = fa.rotary_inv_freq(d)
    fa.rotary_fwd(q, None, f, out=(q, None))
    pos = torch.arange(n - 64, n, dtype=torch.int32, device="cuda")
    want = fa.rotary_fwd(tail[None], None, f, positions=pos)[0]
    assert torch.equal(q[0, -2:, -64:], want[0])
