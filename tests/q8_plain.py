"""Plain 64-bit implementations of the 8-bit key/value cache's writer and reader, and the inputs
its tests use. Attention over the cache is the paged oracle on the values the codes stand for."""
import numpy as np


def e4m3_values():
    """The 256 e4m3 values, by code (4 exponent bits of bias 7, 3 mantissa bits; 0x7F and 0xFF are
    NaN; no infinities)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where(c & 0x80, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


VALUES = e4m3_values()
_POS = VALUES[:127]  # 0 .. 448, ascending


def to_code(y):
    """Nearest e4m3 code (ties to the even code), NaN -> 0x7F; |y| <= 448 otherwise."""
    y = np.asarray(y, np.float64)
    a = np.where(np.isnan(y), 0, np.abs(y))
    assert (a <= 448).all()
    hi = np.minimum(np.searchsorted(_POS, a), 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(y), c | 0x80, c)
    return np.where(np.isnan(y), 0x7F, c).astype(np.uint8)


def block_scale(amax):
    """The smallest 2^k, k >= -100, with amax <= 448 * 2^k."""
    k = -100
    while amax > 448 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def write(codes, scales, x, table, lengths, block):
    """Writes x (a list over sequences of [Hk, n, d] float64 arrays) into codes [P, Hk, ps, d]
    (uint8) and scales [P, Hk, ps / block], in place."""
    P, Hk, ps, _ = codes.shape
    for b, length in enumerate(lengths):
        n = x[b].shape[1]
        if length < 0 or length > table.shape[1] * ps:
            continue
        first = length - n
        lo = max(first, 0)
        if n == 0 or lo >= length:
            continue
        for blk in range(lo // block, (length - 1) // block + 1):
            p0 = blk * block
            new = np.arange(max(p0, lo), min(p0 + block, length))
            old = np.arange(p0, max(p0, lo))
            pg, slot = table[b, p0 // ps], p0 % ps
            if not 0 <= pg < P:
                continue
            for h in range(Hk):
                rows = x[b][h, new - first]
                fine = rows[np.isfinite(rows)]
                s = block_scale(np.abs(fine).max() if fine.size else 0.0)
                if old.size:
                    was = float(scales[pg, h, slot // block])
                    s = max(s, was)
                    if s > was:
                        kept = VALUES[codes[pg, h, old % ps]]
                        codes[pg, h, old % ps] = to_code(kept * (was / s))
                scales[pg, h, slot // block] = s
                codes[pg, h, new % ps] = to_code(np.where(np.isfinite(rows), rows / s, np.nan))


def values(codes, scales):
    """What the codes stand for, in 64 bits."""
    block = codes.shape[2] // scales.shape[2]
    return VALUES[codes] * np.repeat(scales.astype(np.float64), block, axis=2)[..., None]


def make_table(rng, B, per, spare=3):
    pages = rng.permutation(B * per + spare).astype(np.int32)
    return pages[:B * per].reshape(B, per).copy(), B * per + spare


def make_cache(rng, P, Hk, ps, d, block, spread=1.0, sink=False):
    """Random codes and scales of a cache (no NaN codes): (k, v, k_scale, v_scale)."""
    out = []
    for _ in range(2):
        c = to_code(np.clip(rng.standard_normal((P, Hk, ps, d)) * 60, -448, 448))
        out.append(c)
    for _ in range(2):
        out.append((2.0 ** -6 * np.exp(spread * rng.standard_normal((P, Hk, ps // block))))
                   .astype(np.float32))
    return out
