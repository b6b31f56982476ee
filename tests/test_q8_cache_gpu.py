"""The 8-bit key/value cache on the GPU: the writer and the reader bit for bit against a plain
64-bit implementation (every rounding in them is a single one of an exact value, so there is no
tolerance), and attention over the cache against the paged oracle on the values the codes stand
for.

Tolerances of the attention, per element. O is rounded to bf16 (2^-8 of |o|) and each softmax
weight is held to 9 bits (at most 2^-9 of itself, against sum_j p_j |v_j|); the f32 arithmetic in
between (sums of up to 2^14 terms, exponentials good to 2^-22, scores of at most ~2^6 in base 2
rounded to 2^-24 of themselves) stays below 2^-14 of the same sum. L: the f32 score and sum, below
2^-17 of max(1, |L|) by the same count.
"""
import numpy as np
import pytest

import oracle
from tests import q8_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import flash_attention_gb300 as fa

    fa.build()
    oracle.build()
    fa.fa_device_status(True)
    yield
    fa.fa_device_status(True)


def dev_cache(codes_k, codes_v, ks, vs):
    import torch

    c = [torch.from_numpy(x.copy()).cuda().view(torch.float8_e4m3fn) for x in (codes_k, codes_v)]
    return (*c, *(torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda() for x in (ks, vs)))


def ints(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def host_codes(t):
    import torch

    return t.view(torch.uint8).cpu().numpy()


def bf16(x):
    """(CUDA bf16 tensor, its values in 64 bits) of a float array."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().cuda()
    return t, t.double().cpu().numpy()


# ------------------------------------------------------------------------------- writer
WRITES = [
    # name, Hk, d, page, block, lengths before, new rows of each sequence
    ("one_token", 2, 128, 16, 16, [0, 1, 15, 16, 37], [1] * 5),
    ("one_token_d64", 3, 64, 64, 32, [0, 31, 32, 100], [1] * 4),
    ("one_token_d256", 1, 256, 8, 8, [0, 7, 8, 9], [1] * 4),
    ("four_tokens", 2, 128, 32, 32, [0, 29, 30, 31, 64], [4] * 5),
    ("ragged", 2, 128, 16, 16, [0, 3, 0, 50, 16], [33, 0, 1, 17, 300]),
    ("ragged_d64_token_scales", 2, 64, 8, 1, [5, 0, 0], [1, 70, 129]),
    ("ragged_d64_block2", 1, 64, 8, 2, [3, 0], [4, 41]),
    ("ragged_d64_block8", 2, 64, 16, 8, [3, 8, 0], [4, 41, 200]),
    ("ragged_d128_block4", 2, 128, 16, 4, [3, 8, 0], [4, 41, 200]),
    ("ragged_d128_block8", 2, 128, 16, 8, [3, 8, 0], [4, 41, 200]),
    ("ragged_d256_block1", 2, 256, 16, 1, [3, 8, 0], [4, 41, 20]),
    ("ragged_d256_block2", 2, 256, 16, 2, [3, 8, 0], [4, 41, 20]),
    ("wide_block_d128", 2, 128, 256, 256, [0, 255, 256, 300], [5, 3, 700, 1]),
    ("wide_block_d256", 1, 256, 256, 256, [0, 130], [1, 300]),
    ("wide_block_d64", 1, 64, 256, 128, [0, 130], [1, 300]),
    ("many_sequences", 1, 64, 16, 16, [0] * 70, list(range(70))),
]


@pytest.mark.parametrize("layout", ["heads", "rows", "fused"])
@pytest.mark.parametrize("case", WRITES, ids=lambda c: c[0])
def test_write_matches_the_definition(case, layout):
    import torch

    import flash_attention_gb300 as fa

    name, Hk, d, ps, block, past, new = case
    rng = np.random.default_rng(len(name) * 7 + d)
    B, total = len(past), sum(new)
    lengths = np.array(past) + new
    per = int(-(-lengths.max() // ps)) + 1
    table, P = plain.make_table(rng, B, per)
    cache = plain.make_cache(rng, P, Hk, ps, d, block)
    for i in (2, 3):  # powers of two and others
        cache[i][::2] = 2.0 ** np.round(np.log2(cache[i][::2]))
    got = dev_cache(*cache)
    fixed = len(set(new)) == 1
    xs, ts = [], []
    for _ in range(2):
        x = rng.standard_normal((total, Hk, d)) * np.exp(1.5 * rng.standard_normal((total, Hk, 1)))
        x[rng.random((total, Hk)) < 0.05] = 0
        x[rng.random(x.shape) < 0.001] = rng.choice([np.inf, -np.inf, np.nan, -0.0, 1e-40, 3e38])
        t, x = bf16(x)
        if layout == "heads":
            t = t.transpose(0, 1).contiguous()  # [Hk, total, d]
        elif layout == "rows":
            t = t.transpose(0, 1)  # a view of [total, Hk, d]
        else:  # columns of a wider projection
            wide = torch.full((total, Hk * d + 64), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, 64:] = t.reshape(total, -1)
            t = wide[:, 64:].view(total, Hk, d).transpose(0, 1)
        if fixed:  # [B, Hk, n, d]
            t = t.unflatten(1, (B, new[0])).transpose(0, 1)
        xs.append(x)
        ts.append(t)
    cu = np.concatenate([[0], np.cumsum(new)])
    fa.q8_cache_write(*ts, *got, ints(table), ints(lengths), cu_seqlens=None if fixed else ints(cu))
    assert fa.fa_device_status(True) == fa.FA_OK
    for i in range(2):
        x = [xs[i][cu[b]:cu[b + 1]].transpose(1, 0, 2) for b in range(B)]
        plain.write(cache[i], cache[2 + i], x, table, lengths, block)
        np.testing.assert_array_equal(host_codes(got[i]), cache[i])
        np.testing.assert_array_equal(got[2 + i].cpu().numpy(), cache[2 + i])


def test_write_token_by_token_keeps_a_monotone_scale():
    """Tokens that grow by far within one block: earlier codes are rounded again each time."""
    import flash_attention_gb300 as fa

    rng = np.random.default_rng(5)
    Hk, d, ps, block = 2, 64, 16, 16
    table, P = plain.make_table(rng, 1, 2)
    cache = plain.make_cache(rng, P, Hk, ps, d, block)
    got = dev_cache(*cache)
    for i in range(20):
        x = [bf16(rng.standard_normal((1, Hk, 1, d)) * 4.0 ** (i % 7 + i // 4)) for _ in range(2)]
        fa.q8_cache_write(x[0][0], x[1][0], *got, ints(table), ints([i + 1]))
        for w in range(2):
            plain.write(cache[w], cache[2 + w], [x[w][1][0]], table, [i + 1], block)
            np.testing.assert_array_equal(host_codes(got[w]), cache[w])
            np.testing.assert_array_equal(got[2 + w].cpu().numpy(), cache[2 + w])


@pytest.mark.parametrize("d,ps,block", [(64, 256, 256), (128, 256, 256), (256, 256, 256),
                                        (128, 256, 32), (128, 16, 16), (64, 8, 4)])
@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** 12])
def test_write_into_a_block_with_another_scale(d, ps, block, size):
    """New tokens far smaller than a block's earlier ones keep its scale, far larger ones raise it,
    wherever in the block they begin."""
    import flash_attention_gb300 as fa

    rng = np.random.default_rng(d + ps + block)
    past = [1, block // 2, block - 1, block + 3, 2 * block + block // 4]
    new = [3 * block + 1, block, 1, 2, block]
    lengths = np.array(past) + new
    per = int(-(-lengths.max() // ps))
    table, P = plain.make_table(rng, 5, per)
    cache = plain.make_cache(rng, P, 2, ps, d, block, spread=0.3)
    got = dev_cache(*cache)
    cu = np.concatenate([[0], np.cumsum(new)])
    x = [bf16(rng.standard_normal((2, cu[-1], d)) * size) for _ in range(2)]
    fa.q8_cache_write(x[0][0], x[1][0], *got, ints(table), ints(lengths), cu_seqlens=ints(cu))
    for w in range(2):
        plain.write(cache[w], cache[2 + w], [x[w][1][:, cu[b]:cu[b + 1]] for b in range(5)], table,
                    lengths, block)
        np.testing.assert_array_equal(host_codes(got[w]), cache[w])
        np.testing.assert_array_equal(got[2 + w].cpu().numpy(), cache[2 + w])


def test_write_every_bf16_value_rounds_once():
    """All finite bf16 values of one binade range as single-token blocks: the scale is the smallest
    power of two that fits, at the border 448 * 2^k too."""
    import torch

    import flash_attention_gb300 as fa

    bits = np.arange(0, 0x7F80, dtype=np.uint16)
    n = bits.size
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    k = torch.zeros(1, n, 64, dtype=torch.bfloat16, device="cuda")
    k[0, :, 5] = x
    k[0, :, 9] = -x / 3
    ps = 128
    per = -(-n // ps)
    cache = fa.make_q8_cache(per, 1, ps, 64, 1)
    fa.q8_cache_write(k, k, *cache, ints(np.arange(per)[None]), ints([n]),
                      cu_seqlens=ints([0, n]))
    v = k[0].double().cpu().numpy()
    s = np.array([plain.block_scale(a) for a in np.abs(v).max(1)])
    np.testing.assert_array_equal(cache[2].cpu().numpy().reshape(-1)[:n], s)
    want = plain.to_code(v / s[:, None])
    np.testing.assert_array_equal(host_codes(cache[0]).reshape(-1, 64)[:n], want)


def test_write_padded_entries_and_short_lengths():
    """A length of 0 writes nothing; a length below the new rows keeps the last of them."""
    import flash_attention_gb300 as fa

    rng = np.random.default_rng(8)
    Hk, d, ps, block = 2, 128, 16, 8
    table, P = plain.make_table(rng, 3, 2)
    cache = plain.make_cache(rng, P, Hk, ps, d, block)
    got = dev_cache(*cache)
    x = [bf16(rng.standard_normal((3, Hk, 4, d))) for _ in range(2)]
    lengths = [0, 2, 9]
    fa.q8_cache_write(x[0][0], x[1][0], *got, ints(table), ints(lengths))
    assert fa.fa_device_status(True) == fa.FA_OK
    for w in range(2):
        plain.write(cache[w], cache[2 + w], list(x[w][1]), table, lengths, block)
        np.testing.assert_array_equal(host_codes(got[w]), cache[w])
        np.testing.assert_array_equal(got[2 + w].cpu().numpy(), cache[2 + w])


def test_write_out_of_range_inputs_are_flagged_and_left_out():
    import flash_attention_gb300 as fa

    rng = np.random.default_rng(9)
    Hk, d, ps, block = 2, 128, 16, 16
    table, P = plain.make_table(rng, 4, 2)
    cache = plain.make_cache(rng, P, Hk, ps, d, block)
    x = [bf16(rng.standard_normal((4, Hk, 20, d))) for _ in range(2)]
    for lengths, at in (([20, 33, -1, 20], None), ([20, 20, 20, 20], (1, 0)),
                        ([20, 20, 20, 32], (3, 1))):
        t = table.copy()
        if at:
            t[at] = P + 2 if at[1] else -7
        want, got = [c.copy() for c in cache], dev_cache(*cache)
        fa.q8_cache_write(x[0][0], x[1][0], *got, ints(t), ints(lengths))
        assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
        for w in range(2):
            plain.write(want[w], want[2 + w], list(x[w][1]), t, lengths, block)
            np.testing.assert_array_equal(host_codes(got[w]), want[w])
            np.testing.assert_array_equal(got[2 + w].cpu().numpy(), want[2 + w])
    # offsets out of range are clamped to the rows there are, and flagged
    got = dev_cache(*cache)
    k = x[0][0][0]
    for cu in ([0, 5, 9, 15, 40], [0, 9, 5, 15, 20], [-3, 5, 9, 15, 20]):
        fa.q8_cache_write(k, k, *got, ints(table), ints([20] * 4), cu_seqlens=ints(cu))
        assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT


# ------------------------------------------------------------------------------- reader
READS = [
    ("d128", 2, 128, 16, 16, [37, 0, 1, 16, 300]),
    ("d64_token_scales", 3, 64, 8, 1, [5, 129]),
    ("d256", 1, 256, 32, 8, [33, 64]),
    ("d64_wide_page", 1, 64, 256, 256, [500, 3]),
    ("many", 1, 64, 16, 16, list(range(70))),
]


@pytest.mark.parametrize("case", READS, ids=lambda c: c[0])
def test_read_matches_the_definition(case):
    import torch

    import flash_attention_gb300 as fa

    name, Hk, d, ps, block, lens = case
    rng = np.random.default_rng(len(name) + 40)
    per = max(1, -(-max(lens) // ps))
    table, P = plain.make_table(rng, len(lens), per)
    cache = plain.make_cache(rng, P, Hk, ps, d, block)
    cache[0][table[0, 0], :, 1] = np.arange(d) % 256  # every code, NaN among them
    got = dev_cache(*cache)
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1]) + 7  # rows behind the last sequence stay as they are
    fill = torch.full((total, 2, Hk, d), 7.0, dtype=torch.bfloat16, device="cuda")
    outs = [tuple(torch.full((Hk, total, d), 7.0, dtype=torch.bfloat16, device="cuda")
                  for _ in range(2)), tuple(fill[:, w].transpose(0, 1) for w in range(2))]
    for out in outs:
        k, v = fa.q8_cache_read(*got, ints(table), ints(cu), total, out=out)
        assert fa.fa_device_status(True) == fa.FA_OK
        for w, t in enumerate((k, v)):
            val = plain.values(cache[w], cache[2 + w]).astype(np.float32)
            want = torch.full((Hk, total, d), 7.0, dtype=torch.bfloat16)
            for b, n in enumerate(lens):
                j = np.arange(n)
                rows = val[table[b, j // ps], :, j % ps].transpose(1, 0, 2)
                want[:, cu[b]:cu[b + 1]] = torch.from_numpy(rows).bfloat16()
            assert torch.equal(torch.nan_to_num(t.cpu().float(), nan=1e9),
                               torch.nan_to_num(want.float(), nan=1e9))
    k, v = fa.q8_cache_read(*got, ints(table), ints(cu), int(cu[-1]))
    assert k.shape == (Hk, cu[-1], d) and torch.equal(
        torch.nan_to_num(k.float(), nan=1e9),
        torch.nan_to_num(outs[0][0][:, :cu[-1]].float(), nan=1e9))


def test_read_out_of_range_inputs_read_as_zeros():
    import flash_attention_gb300 as fa

    rng = np.random.default_rng(11)
    table, P = plain.make_table(rng, 2, 2)
    cache = dev_cache(*plain.make_cache(rng, P, 2, 16, 64, 16))
    good = fa.q8_cache_read(*cache, ints(table), ints([0, 20, 40]), 40)
    table[1, 0] = P
    k, v = fa.q8_cache_read(*cache, ints(table), ints([0, 20, 40]), 40)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    assert (k[:, 20:36] == 0).all() and (v[:, 20:36] == 0).all()
    assert (k[:, :20] == good[0][:, :20]).all() and (k[:, 36:] == good[0][:, 36:]).all()
    k, v = fa.q8_cache_read(*cache, ints(table[:1]), ints([0, 40]), 40)  # past the table's end
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    assert (k[:, 32:] == 0).all() and (k[:, :20] == good[0][:, :20]).all()


# ---------------------------------------------------------------------------- attention
def A(name, B, H, Hk, lq, d, ps, block, lengths, causal=True):
    return dict(name=name, B=B, H=H, Hk=Hk, lq=lq, d=d, ps=ps, block=block, lengths=lengths,
                causal=causal)


ATTEND = [
    A("one_key", 1, 4, 4, 1, 128, 16, 16, [1]),
    A("short", 1, 4, 4, 1, 128, 16, 16, [37]),
    A("tile_edges", 6, 8, 2, 1, 128, 16, 16, [127, 128, 129, 255, 256, 257]),
    A("d64_page8_token_scales", 3, 4, 2, 1, 64, 8, 1, [5, 130, 700]),
    A("d64_mha", 4, 3, 3, 1, 64, 64, 32, [1, 64, 300, 1000]),
    A("d256_page8", 2, 8, 2, 1, 256, 8, 4, [9, 513]),
    A("d256_gqa16", 2, 16, 1, 1, 256, 32, 8, [300, 1100]),
    A("d256_rows32", 1, 32, 1, 1, 256, 64, 64, [700]),
    A("gqa8", 3, 16, 2, 1, 128, 32, 32, [1, 64, 300]),
    A("gqa16_rows", 2, 32, 2, 1, 128, 128, 32, [200, 1500]),
    A("gqa32_rows", 1, 32, 1, 1, 128, 256, 256, [1500]),
    A("lq4", 2, 8, 2, 4, 128, 16, 16, [4, 77]),
    A("lq5_odd_rows", 3, 6, 2, 5, 64, 16, 8, [5, 130, 260]),
    A("lq33_several_row_blocks", 2, 4, 2, 33, 128, 32, 16, [33, 400]),
    A("lq130_past_its_length", 2, 2, 1, 130, 64, 16, 16, [100, 500]),
    A("lq40_d256", 1, 4, 2, 40, 256, 16, 16, [90]),
    A("noncausal_lq3", 2, 4, 2, 3, 128, 16, 16, [40, 200], causal=False),
    A("lq_gt_len", 2, 4, 2, 6, 64, 8, 8, [3, 50]),
    A("empty_sequences", 4, 4, 2, 1, 128, 16, 16, [0, 90, 0, 0]),
    A("all_empty", 2, 4, 2, 2, 128, 16, 16, [0, 0]),
    A("long", 2, 8, 2, 1, 128, 16, 16, [5000, 3000]),
    A("one_long", 1, 1, 1, 1, 128, 256, 256, [16000]),
    A("very_long", 1, 2, 1, 1, 64, 64, 16, [150_001]),
    A("many_short", 100, 4, 2, 1, 64, 16, 4, [(i * 37) % 200 for i in range(100)]),
]


def make_attend(c, seed=0, spread=0.7):
    rng = np.random.default_rng(seed + 100 + c["d"] + c["lq"] + sum(c["lengths"]))
    per = max(1, -(-max(c["lengths"]) // c["ps"]))
    table, P = plain.make_table(rng, c["B"], per)
    cache = plain.make_cache(rng, P, c["Hk"], c["ps"], c["d"], c["block"], spread)
    q = rng.standard_normal((c["B"], c["H"], c["lq"], c["d"]))
    return rng, table, P, cache, q


def poison(c, table, cache):
    """NaN codes and NaN scales wherever no sequence has a key."""
    k, v, ks, vs = [x.copy() for x in cache]
    used = np.zeros(k.shape[:1] + k.shape[2:3], bool)  # [P, ps]
    for b, n in enumerate(c["lengths"]):
        j = np.arange(n)
        used[table[b, j // c["ps"]], j % c["ps"]] = True
    for x in (k, v):
        x[~used[:, None].repeat(c["Hk"], 1)] = 0x7F
    free = ~used.reshape(used.shape[0], -1, c["block"]).any(2)
    for s in (ks, vs):
        s[free[:, None].repeat(c["Hk"], 1)] = np.nan
    return k, v, ks, vs


def check_attend(c, table, cache, q, o, lse):
    """o, lse (tensors) against the oracle; returns the largest shares of the tolerances used."""
    kv = [np.nan_to_num(plain.values(cache[w], cache[2 + w]), nan=0.0) for w in range(2)]
    kw = dict(scale=c["d"] ** -0.5, causal=c["causal"])
    want, l_want = oracle.paged_fwd(q, kv[0], kv[1], table, np.array(c["lengths"]), **kw)
    mass, _ = oracle.paged_fwd(q, kv[0], np.abs(kv[1]), table, np.array(c["lengths"]), **kw)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    dead = np.isneginf(l_want)
    assert (np.isneginf(lse) == dead).all() and (o[dead] == 0).all()
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -14) * mass + 1e-30
    used = np.max(np.abs(o - want) / tol)
    l_used = 0.0
    if not dead.all():
        d = np.abs(lse[~dead] - l_want[~dead]) / np.maximum(1, np.abs(l_want[~dead]))
        l_used = float(np.max(d) * 2 ** 17)
    assert used <= 1 and l_used <= 1, (c["name"], used, l_used)
    return used, l_used


def attend(c, table, cache, q, **kw):
    import flash_attention_gb300 as fa

    return fa.q8_paged_attention(q, *cache, ints(table), ints(c["lengths"]),
                                 scale=c["d"] ** -0.5, causal=c["causal"], **kw)


@pytest.mark.parametrize("c", ATTEND, ids=lambda c: c["name"])
def test_attention_matches_the_oracle(c):
    import flash_attention_gb300 as fa

    _, table, P, cache, q = make_attend(c)
    qt, q = bf16(q)
    o, lse = attend(c, table, dev_cache(*poison(c, table, cache)), qt)
    assert fa.fa_device_status(True) == fa.FA_OK
    print(c["name"], check_attend(c, table, cache, q, o, lse))


@pytest.mark.parametrize("name", ["peak", "sink", "scales", "tiny", "large", "rising"])
def test_attention_with_uneven_softmax_and_scales(name):
    """One key that takes nearly all of the weight; the same with next to nothing behind it (what
    counts is spread over thousands of small weights); value scales over 2^40; tiny and large
    queries; scores that rise from tile to tile (the running maximum moves all the time)."""
    import flash_attention_gb300 as fa

    c = A(name, 2, 4, 2, 1, 128, 16, 1 if name != "peak" else 16, [3000, 4500])
    rng, table, P, cache, q = make_attend(c)
    if name in ("peak", "sink"):
        q[:] = 1.0
        for b in range(2):
            cache[0][table[b, 3], :, 5] = plain.to_code(np.full(128, 24.0))
            cache[2][table[b, 3], :, 5 if name == "sink" else 0] = 2.0 ** -4
        cache[0][:] = np.where(np.arange(16)[:, None] % 16 == 5, cache[0],
                               plain.to_code(plain.VALUES[cache[0]] / 64))
        if name == "sink":  # its value is small, the others have a common part
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


def test_attention_out_of_range_inputs_are_flagged_not_faulted():
    import torch

    import flash_attention_gb300 as fa

    c = A("bad", 2, 4, 2, 1, 128, 16, 16, [50, 100])
    _, table, P, cache, q = make_attend(c)
    qt, _ = bf16(q)
    got = dev_cache(*cache)
    bad = dict(c, lengths=[5000, 100])  # clamped to the table's capacity
    attend(bad, table, got, qt)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    attend(dict(c, lengths=[-4, 100]), table, got, qt)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    t = table.copy()
    t[1, 0], t[1, 1] = P + 7, -3  # pages outside the cache read as zero keys and values
    o, lse = attend(c, t, got, qt)
    assert fa.fa_device_status(True) == fa.FA_ERR_BAD_INPUT
    zero = [np.concatenate([x, np.zeros_like(x[:1]) + (i > 1)]) for i, x in enumerate(cache)]
    t[1, 0] = t[1, 1] = P
    _, q64 = bf16(q)
    check_attend(c, t, zero, q64, o, lse)
    o, lse = attend(c, table, got, qt)
    assert fa.fa_device_status(True) == fa.FA_OK and torch.isfinite(o.float()).all()


def test_attention_nan_stays_in_its_rows():
    """A query row that is not finite gives NaN there and nowhere else; so does a NaN code that a
    row sees, in its head alone."""
    import torch

    c = A("nan", 2, 8, 2, 1, 128, 16, 16, [300, 200])
    _, table, P, cache, q = make_attend(c)
    qt, _ = bf16(q)
    o0, l0 = attend(c, table, dev_cache(*cache), qt)
    bad = qt.clone()
    bad[0, 1, 0, 7] = float("nan")
    bad[1, 6, 0, 9] = float("inf")
    o, lse = attend(c, table, dev_cache(*cache), bad)
    hit = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 6] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(o[~hit], o0[~hit]) and torch.equal(lse[~hit], l0[~hit])
    cache[1][table[1, 2], 1, 3, 5] = 0x7F  # a value of sequence 1, kv head 1
    o, lse = attend(c, table, dev_cache(*cache), qt)
    hit = torch.zeros(2, 8, 1, 128, dtype=torch.bool, device="cuda")
    hit[1, 4:, 0, 5] = True
    assert torch.equal(o.isnan(), hit) and torch.equal(lse, l0)


@pytest.mark.parametrize("d,H,lq", [(128, 8, 3), (64, 2, 5), (256, 8, 4)])
def test_attention_nan_behind_a_row_does_not_reach_it(d, H, lq):
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


def test_attention_is_bitwise_reproducible():
    import torch

    c = A("again", 5, 8, 2, 2, 128, 16, 16, [5, 900, 0, 2500, 131])
    _, table, P, cache, q = make_attend(c)
    got = dev_cache(*cache)
    qt, _ = bf16(q)
    first = attend(c, table, got, qt)
    for _ in range(5):
        again = attend(c, table, got, qt)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_attention_writes_its_outputs_and_nothing_else():
    """Through the C ABI, with o and lse inside filled buffers: every element of them is written, and
    none around them, for whole and cut units, empty sequences and head dims of every width."""
    import ctypes

    import torch

    import flash_attention_gb300 as fa

    for d, lq, lengths in ((64, 1, [5, 0, 900]), (128, 3, [2000, 1, 0]), (256, 5, [300, 0, 700])):
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


def test_caches_beyond_32_bits():
    """The last pages of caches of over 4 GB, against the same pages in a small cache."""
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(31)
    Hk, ps, d, block, B = 8, 16, 128, 4, 3
    lengths = [200, 33, 130]
    table, P = plain.make_table(rng, B, 13)
    small = fa.make_q8_cache(P, Hk, ps, d, block)
    big_pages = (1 << 32) // (Hk * ps * d) + P
    big = (*(torch.empty((big_pages, Hk, ps, d), dtype=torch.uint8, device="cuda")
             .view(torch.float8_e4m3fn) for _ in range(2)),
           *(torch.empty((big_pages, Hk, ps // block), device="cuda") for _ in range(2)))
    off = big_pages - P
    cu = np.concatenate([[0], np.cumsum(lengths)])
    x = [bf16(rng.standard_normal((Hk, cu[-1], d)))[0] for _ in range(2)]
    q = bf16(rng.standard_normal((B, 16, 1, d)))[0]
    got = []
    for cache, t in ((small, table), (big, table + off)):
        fa.q8_cache_write(*x, *cache, ints(t), ints(lengths), cu_seqlens=ints(cu))
        got.append((*fa.q8_cache_read(*cache, ints(t), ints(cu), int(cu[-1])),
                    *fa.q8_paged_attention(q, *cache, ints(t), ints(lengths), scale=0.1)))
    assert fa.fa_device_status(True) == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_attention_waits_that_run_out_are_reported():
    """With a limit of 1 ns the kernel's ordinary waits run out: it winds down, the status says so,
    and with the default limit the same calls are right again."""
    import flash_attention_gb300 as fa

    cases = [A("long", 2, 8, 2, 1, 128, 16, 16, [5000, 3000]),
             A("rows16", 3, 16, 2, 2, 64, 16, 16, [500, 100, 1]),
             A("d256", 2, 4, 2, 3, 256, 32, 8, [700, 300])]
    for c in cases:
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


# ------------------------------------------------------------------- together, and captured
def test_prompt_then_decode_as_a_server_runs_it():
    """A packed batch of prompts is written, then every step writes one token a sequence and
    attends; the prompt's last rows attend over what is cached through the packed training
    attention on the read-back keys too. Checked against the plain cache and the oracle."""
    import torch

    import flash_attention_gb300 as fa

    rng = np.random.default_rng(21)
    B, H, Hk, d, ps, block = 3, 8, 2, 128, 16, 8
    prompts = [40, 1, 133]
    per = 12
    table, P = plain.make_table(rng, B, per)
    cache = [np.zeros((P, Hk, ps, d), np.uint8), np.zeros((P, Hk, ps, d), np.uint8),
             np.ones((P, Hk, ps // block), np.float32), np.ones((P, Hk, ps // block), np.float32)]
    got = fa.make_q8_cache(P, Hk, ps, d, block)
    cu = np.concatenate([[0], np.cumsum(prompts)])
    tb = ints(table)

    def both(x, lengths, **kw):
        fa.q8_cache_write(x[0][0], x[1][0], *got, tb, ints(lengths), **kw)

    x = [bf16(rng.standard_normal((Hk, cu[-1], d))) for _ in range(2)]
    both(x, prompts, cu_seqlens=ints(cu))
    for w in range(2):
        plain.write(cache[w], cache[2 + w], [x[w][1][:, cu[b]:cu[b + 1]] for b in range(B)],
                    table, prompts, block)
    # the prompt's own attention over the cached keys, packed
    q = bf16(rng.standard_normal((H, cu[-1], d)))[0]
    k, v = fa.q8_cache_read(*got, tb, ints(cu), int(cu[-1]))
    o, _ = fa.varlen_attention_fwd(q, k, v, ints(cu), ints(cu), 133, 133, scale=d ** -0.5,
                                   causal=True)
    c = A("prompt", 1, H, Hk, 133, d, ps, block, [133])
    o2, l2 = fa.q8_paged_attention(q[:, cu[2]:].unsqueeze(0).contiguous(), *got, tb[2:],
                                   ints([133]), scale=d ** -0.5)
    check_attend(c, table[2:], cache, q[:, cu[2]:].double().cpu().numpy()[None], o2, l2)
    assert (o[:, cu[2]:].float() - o2[0].float()).abs().max() < 0.05
    lengths = np.array(prompts)
    for step in range(10):
        lengths += 1
        x = [bf16(rng.standard_normal((B, Hk, 1, d)) * (1 + step)) for _ in range(2)]
        both(x, lengths)
        for w in range(2):
            plain.write(cache[w], cache[2 + w], list(x[w][1]), table, lengths, block)
        qt, q64 = bf16(rng.standard_normal((B, H, 1, d)))
        c = A("step", B, H, Hk, 1, d, ps, block, lengths.tolist())
        o, lse = attend(c, table, got, qt)
        check_attend(c, table, cache, q64, o, lse)
    for w in range(2):
        np.testing.assert_array_equal(host_codes(got[w]), cache[w])
        np.testing.assert_array_equal(got[2 + w].cpu().numpy(), cache[2 + w])
    assert fa.fa_device_status(True) == fa.FA_OK


def test_calls_on_another_stream_and_in_graphs():
    """Two decoding graphs captured and replayed on one stream after the other, with lengths that
    grow between replays, equal the eager calls; so do calls given a stream of their own."""
    import torch

    import flash_attention_gb300 as fa

    c = A("graph", 4, 8, 2, 1, 128, 16, 16, [30, 700, 1, 250])
    rng, table, P, cache, q = make_attend(dict(c, lengths=[60, 730, 40, 280]))
    tb = ints(table)

    def state():
        return dict(cache=dev_cache(*cache), lens=ints(c["lengths"]),
                    q=bf16(q)[0], kv=bf16(rng0.standard_normal((2, 4, 2, 1, 128)))[0])

    def step(s, stream=None):
        s["lens"] += 1
        if stream is not None:
            torch.cuda.synchronize()
        fa.q8_cache_write(s["kv"][0], s["kv"][1], *s["cache"], tb, s["lens"], stream=stream)
        return fa.q8_paged_attention(s["q"], *s["cache"], tb, s["lens"], scale=0.1, stream=stream)

    want = []
    rng0 = np.random.default_rng(3)
    s = state()
    for _ in range(6):
        want.append(step(s))
    torch.cuda.synchronize()
    rng0 = np.random.default_rng(3)
    s = state()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s))
        graphs.append(g)
    for i in range(6):
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for x, y in zip(outs[i % 2], want[i]):
            assert torch.equal(x, y)
    rng0 = np.random.default_rng(3)
    s = state()
    side = torch.cuda.Stream()
    for i in range(6):
        got = step(s, stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[i]))


def test_two_streams_at_once():
    import torch

    import flash_attention_gb300 as fa

    c = A("streams", 4, 8, 2, 1, 128, 16, 16, [3000, 700, 1, 250])
    _, table, P, cache, q = make_attend(c)
    got, tb, lens = dev_cache(*cache), ints(table), ints(c["lengths"])
    qs = [bf16(q * s)[0] for s in (1.0, 0.5)]
    want = [fa.q8_paged_attention(x, *got, tb, lens, scale=0.1) for x in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [fa.q8_paged_attention(x, *got, tb, lens, scale=0.1, stream=s)
                for x, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert fa.fa_device_status(True) == fa.FA_OK


FIRST_CALLS = """
import torch
import flash_attention_gb300 as fa

B, Hk, d, ps = 2, 2, 128, 16
table = torch.randperm(80, device="cuda").to(torch.int32).view(B, 40).contiguous()
lens = torch.tensor([300, 600], device="cuda", dtype=torch.int32)
cu = torch.tensor([0, 300, 900], device="cuda", dtype=torch.int32)
x = torch.randn(2, Hk, 900, d, device="cuda").bfloat16()
q = [torch.randn(B, 8, n, d, device="cuda").bfloat16() for n in (1, 16)]
cache = fa.make_q8_cache(80, Hk, ps, d)


def step():
    out = []
    fa.q8_cache_write(x[0], x[1], *cache, table, lens, cu_seqlens=cu)
    for y in q:
        out += fa.q8_paged_attention(y, *cache, table, lens, scale=0.1)
    return out + list(fa.q8_cache_read(*cache, table, cu, 900))


torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and fa.fa_device_status(True) == 0
"""


def test_a_process_whose_first_calls_are_captured():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
