"""Plain 64-bit implementations of a drafted decoding step's operators (rotary positions, appending
to a paged cache, attention of a tree, keeping accepted nodes), in NumPy, and their tests' inputs."""
import numpy as np


def inv_freq(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def turn(x, pos, freq, interleaved=False, scale=1.0, back=False):
    """x [..., rows, d] float64 turned by the positions pos [..., rows] (broadcast)."""
    a = np.asarray(pos, np.longdouble)[..., None] * np.asarray(freq, np.longdouble)
    c, s = (np.asarray(f(a), np.float64) * scale for f in (np.cos, np.sin))
    s = -s if back else s
    half, y = len(freq), x.copy()
    i = np.arange(half)
    i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    with np.errstate(invalid="ignore"):
        y[..., i1] = x[..., i1] * c - x[..., i2] * s
        y[..., i2] = x[..., i1] * s + x[..., i2] * c
    return y


def turn_bound(x, y, rot, interleaved, scale):
    """How far a turned bf16 element may be from y. One rounding to bf16, 2^-8 of the element; a sine
    and a cosine off by 2^-21 each for what CUDA documents of its fast ones within pi and by as much
    again for the angle's own rounding in 32 bits (2^-24 of pi, twice), and two products and a sum
    rounded in 32 bits: below 2^-19 of scale (|x1| + |x2|)."""
    a, half = np.abs(x), rot // 2
    i = np.arange(half)
    i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    b = np.zeros_like(y)
    b[..., i1] = b[..., i2] = (a[..., i1] + a[..., i2]) * abs(scale) * 2.0 ** -19
    return b + 2.0 ** -8 * np.abs(y) + 2.0 ** -133  # (half a step of the smallest bf16 numbers)


def make_table(rng, B, per, spare=3):
    pages = rng.permutation(B * per + spare).astype(np.int32)
    return pages[:B * per].reshape(B, per).copy(), B * per + spare


def random_trees(rng, B, T, most=5):
    """(ancestors and itself of each node [B, T, T], parents [B, T]): a node's parent is one of the
    few before it, or the sequence itself (-1)."""
    sees = np.zeros((B, T, T), bool)
    parents = np.full((B, T), -1)
    for b in range(B):
        for i in range(T):
            p = i - int(rng.integers(1, most + 1))
            parents[b, i] = max(p, -1)
            if p >= 0:
                sees[b, i] = sees[b, p]
            sees[b, i, i] = True
    return sees, parents


def keys_of(cache, row, n):
    """The first n keys of a sequence [Hk, n, d] from a cache [P, Hk, ps, d]; zeros for pages outside."""
    P, Hk, ps, d = cache.shape
    j = np.arange(n)
    page = row[j // ps] if n else np.zeros(0, int)
    ok = (page >= 0) & (page < P)
    x = cache[np.where(ok, page, 0), :, j % ps]
    return np.where(ok[:, None, None], x, 0.0).transpose(1, 0, 2)


def tree_attention(q, k_cache, v_cache, table, lengths, mask, scale):
    """(o, lse, sum of weight * |v|) of q [B, H, T, d]; mask [B, T, T] or [T, T]."""
    B, H, T, d = q.shape
    Hk, ps = k_cache.shape[1:3]
    o, w = np.zeros((B, H, T, d)), np.zeros((B, H, T, d))
    lse = np.full((B, H, T), -np.inf)
    for b in range(B):
        n = int(np.clip(lengths[b], 0, table.shape[1] * ps))
        k, v = keys_of(k_cache, table[b], n), keys_of(v_cache, table[b], n)
        m = mask if mask.ndim == 2 else mask[b]
        sees = np.ones((T, n), bool)
        sees[:, max(0, n - T):] = m[:, max(0, T - n):]
        for h in range(H):
            for i in range(T):
                at = sees[i]
                if not at.any():
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    s = k[h // (H // Hk)][at] @ q[b, h, i] * scale
                    top = s.max()
                    p = np.exp(s - top)
                    lse[b, h, i] = top + np.log(p.sum())
                    p /= p.sum()
                    o[b, h, i] = p @ v[h // (H // Hk)][at]
                    w[b, h, i] = p @ np.abs(v[h // (H // Hk)][at])
    return o, lse, w


def append(k_cache, v_cache, ks, vs, table, lengths):
    """Writes ks, vs (lists over sequences of [Hk, n, d]) as each sequence's last positions."""
    P, Hk, ps, d = k_cache.shape
    for b, length in enumerate(lengths):
        n = ks[b].shape[1]
        if length < 0 or length > table.shape[1] * ps:
            continue
        for i in range(n):
            pos = length - n + i
            if pos < 0:
                continue
            page = table[b, pos // ps]
            if 0 <= page < P:
                k_cache[page, :, pos % ps] = ks[b][:, i]
                v_cache[page, :, pos % ps] = vs[b][:, i]


def keep(caches, table, lengths, kept, T):
    """Moves the nodes kept[b] (a list) of each sequence's last T to the front of the T, in place;
    returns the new lengths."""
    new = []
    for b, length in enumerate(lengths):
        base = length - T
        ps = caches[0].shape[2]
        for x in caches:
            rows = {i: x[table[b, (base + n) // ps], :, (base + n) % ps].copy()
                    for i, n in enumerate(kept[b]) if n != i}
            for i, r in rows.items():
                x[table[b, (base + i) // ps], :, (base + i) % ps] = r
        new.append(max(0, base + len(kept[b])))
    return new
