"""The operators of the 8-bit key/value cache as work to be measured: attention over the cache,
quantising new keys and values as they are written to it, and reading a batch's keys and values
back.

The cache holds e4m3 codes in pages, [num_pages, kv_heads, page, dim], with one float32 scale for
each block of `block` positions of a page and each head, [num_pages, kv_heads, page / block]. A
code c with the scale s stands for c * s. Key j of a sequence is in page table[b, j // page], slot
j % page.

  attend: o = softmax(scale * q k^T) v over each sequence's first lengths[b] keys, and the
          natural logarithm of the softmax's sum; the q_len queries are the sequence's last
          positions (query i sees key j iff j <= length - q_len + i)
  write:  the new rows of sequence b become positions length - n .. length - 1. A block's scale is
          the smallest power of two (2^-100 at least) with which its largest finite value fits
          into 448, and never less than the scale of the tokens that the block held already, whose
          codes are rounded again where the scale grows. Values that are not finite become NaN.
  read:   bf16(c * s) of each sequence's first keys, packed head-major without padding

`run` computes them in elementary operations, or with `own` set through the framework's calls.
"""
import random

import torch

own = False

SPARE = 5  # pages of a cache that no sequence uses


def _attend(name, B, H, Hk, d, lq, page, block, lo, hi, lens, causal=True):
    return dict(name=name, op="attend", B=B, H=H, Hk=Hk, d=d, lq=lq, page=page, block=block,
                min_len=lo, max_len=hi, lens=lens, causal=causal)


def _write(name, B, Hk, d, page, block, past, lo, hi, lens):
    return dict(name=name, op="write", B=B, Hk=Hk, d=d, page=page, block=block, past=past,
                min_len=lo, max_len=hi, lens=lens)


def _read(name, B, Hk, d, page, block, lo, hi, lens):
    return dict(name=name, op="read", B=B, Hk=Hk, d=d, page=page, block=block, min_len=lo,
                max_len=hi, lens=lens)


def listed():
    return [
        # one short conversation: the latency of a call
        _attend("attend 1x37", 1, 4, 4, 128, 1, 16, 16, 37, 37, 1),
        # single-query decoding of a server's batch, grouped heads, small pages
        _attend("attend 16x16k", 16, 32, 8, 128, 1, 16, 16, 2048, 16384, 2),
        # four new positions a sequence (speculated tokens), a scale for each token
        _attend("attend 16x16k lq4", 16, 32, 8, 128, 4, 16, 1, 2048, 16384, 3),
        # many short conversations, every head its own keys
        _attend("attend 128x2k d64", 128, 8, 8, 64, 1, 64, 32, 1, 2047, 4),
        # wide heads, odd lengths
        _attend("attend 7x8k d256", 7, 16, 4, 256, 1, 32, 8, 501, 8191, 5),
        # a chunk of 32 prompt tokens against what is cached already
        _attend("attend 5x4k lq32", 5, 32, 8, 128, 32, 64, 64, 33, 4095, 6),
        # the largest decoding batch
        _attend("attend 64x16k", 64, 32, 8, 128, 1, 32, 32, 1024, 16384, 7),
        # the token that each sequence of a decoding batch adds, past its first block
        _write("write 16x1", 16, 8, 128, 16, 16, 16383, 1, 1, 8),
        # a few tokens each for many sequences, a scale for each token
        _write("write 100x33 d64", 100, 8, 64, 64, 1, 500, 1, 33, 9),
        # a batch of prompts of mixed lengths
        _write("write 16x8k", 16, 8, 128, 16, 16, 0, 256, 8192, 10),
        # short sequences read back for a prompt's attention
        _read("read 9x129", 9, 4, 128, 16, 16, 1, 129, 11),
        # a batch of cached prompts of mixed lengths
        _read("read 16x8k", 16, 8, 128, 16, 16, 256, 8192, 12),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("attend", "attend", "write", "read"))
    d = rng.choice((64, 128, 256))
    Hk = rng.choice((1, 2, 4, 8))
    page = rng.choice((8, 16, 32, 64, 128))
    block = rng.choice([b for b in (1, 4, 8, 16, 32, 64, 128) if b <= page])
    B, lens = log(1, 96), rng.randrange(1 << 20)
    most = max(64, min(16384, (1 << 29) // (B * Hk * d)))  # no more than the largest listed case
    hi = log(8, most)
    lo = max(1, hi // rng.choice((1, 2, 30)))
    if op == "attend":
        G, lq = rng.choice((1, 2, 4, 8)), rng.choice((1, 1, 1, 2, 5, 17))
        return dict(op=op, B=B, H=G * Hk, Hk=Hk, d=d, lq=lq, page=page, block=block, min_len=lo,
                    max_len=hi, lens=lens, causal=rng.random() < 0.8)
    if op == "write":
        one = rng.random() < 0.4
        return dict(op=op, B=B, Hk=Hk, d=d, page=page, block=block, past=rng.choice((0, 9, 700)),
                    min_len=1 if one else lo, max_len=1 if one else min(hi, 8192), lens=lens)
    return dict(op=op, B=B, Hk=Hk, d=d, page=page, block=block, min_len=lo, max_len=min(hi, 8192),
                lens=lens)


def _lengths(case):
    """(new or cached rows of each sequence, rows that were there before); the last sequence is
    the longest."""
    r = random.Random(case["lens"])
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["B"])]
    lens[-1] = case["max_len"]
    past = [r.randint(0, case["past"]) for _ in lens] if case["op"] == "write" else [0] * len(lens)
    return lens, past


def work(case):
    lens, past = _lengths(case)
    rows, Hk, d = sum(lens), case["Hk"], case["d"]
    blocks = sum(-(-n // case["block"]) for n in lens)
    kv, scales = rows * Hk * d * 2, blocks * Hk * 4 * 2
    table = 4 * sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "attend":
        q = case["B"] * case["H"] * case["lq"]
        return {"bytes": kv + scales + table + q * (4 * d + 4),
                "flops": 4 * d * case["H"] * case["lq"] * rows}
    return {"bytes": 3 * kv + scales + table, "flops": 2 * rows * Hk * d}


def _power(amax):
    """The smallest power of two s >= 2^-100 with amax <= 448 s (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-100)
    k = torch.where(amax > 0, k, -100)
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x):
    return x.to(torch.float8_e4m3fn)


def _filled(case, g, pages, spread):
    """Codes and scales of a cache whose tokens differ in size and whose keys have a few large
    channels."""
    P, Hk, page, d, block = pages, case["Hk"], case["page"], case["d"], case["block"]
    x = torch.randn(P, Hk, page // block, block, d, generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn(P, 1, page // block, block, 1, generator=g, device="cuda"))
    x *= 1 + 3 * (torch.rand(Hk, 1, 1, d, generator=g, device="cuda") < 0.03)
    s = _power(x.abs().amax((3, 4)))
    return _codes(x / s[..., None, None]).view(P, Hk, page, d), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, past = _lengths(case)
    B, Hk, d, page = case["B"], case["Hk"], case["d"], case["page"]
    total = [n + p for n, p in zip(lens, past)]
    per = -(-max(total) // page)
    pages = B * per + SPARE
    s = dict(case=case, table=torch.randperm(pages, generator=g, device="cuda")[:B * per]
             .view(B, per).int(), lengths=torch.tensor(total, dtype=torch.int32, device="cuda"))
    for n, spread in (("k", 0.25), ("v", 0.5)):
        s[n + "_cache"], s[n + "_scale"] = _filled(case, g, pages, spread)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    if case["op"] == "attend":
        q = torch.randn(B, case["H"], case["lq"], d, generator=g, device="cuda")
        s["q"], s["scale"] = q.bfloat16(), d ** -0.5
    else:
        s["total"] = cu[-1]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "write":
        # one row a sequence comes as a decoding step has it, [B, Hk, 1, d]; others packed
        s["packed"] = case["max_len"] > 1
        shape = (Hk, cu[-1], d) if s["packed"] else (B, Hk, 1, d)
        for n in "kv":
            x = torch.randn(shape, generator=g, device="cuda")
            x *= torch.exp(0.7 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))
            s[n] = x.bfloat16()
    return s


def _values(codes, scale, block):
    """What the codes [..., rows, d] stand for, in the scales' type."""
    return codes.to(scale.dtype) * scale.repeat_interleave(block, -1)[..., None]


def _plain_attend(s):
    c, q, table = s["case"], s["q"], s["table"].long()
    B, H, lq, d = q.shape
    Hk, block = c["Hk"], c["block"]

    def gathered(n):  # [B, pages, Hk, page, d] -> [B, Hk, keys, d]
        x = s[n + "_cache"].view(torch.uint8)[table].view(torch.float8_e4m3fn)
        x = _values(x, s[n + "_scale"][table], block)
        return x.transpose(1, 2).reshape(B, Hk, -1, d)

    k, v = gathered("k"), gathered("v")
    a = torch.matmul(q.float().view(B, Hk, -1, d), k.transpose(2, 3)) * s["scale"]
    a = a.view(B, Hk, H // Hk, lq, -1)
    j = torch.arange(a.shape[-1], device=a.device)
    last = s["lengths"].long()[:, None] - 1 + torch.zeros(lq, dtype=torch.long, device=a.device)
    if c["causal"]:
        last = last - lq + 1 + torch.arange(lq, device=a.device)
    seen = (j <= last[..., None])[:, None, None]  # [B, 1, 1, lq, keys]
    a = torch.where(seen, a, -torch.inf)
    top = a.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(a - top)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, -1, p.shape[-1]), v).view(B, Hk, -1, lq, d)
    o = torch.where(z > 0, o / z, 0.0)
    return {"o": o.reshape(B, H, lq, d).bfloat16(), "lse": (top + z.log()).reshape(B, H, lq)}


def _plain_write(s):
    c = s["case"]
    page, block, table, length = c["page"], c["block"], s["table"].long(), s["lengths"].long()
    cu, nb = s["cu"].long(), page // block
    i = torch.arange(s["total"], device=cu.device)
    b = torch.searchsorted(cu, i, right=True) - 1
    first = length - (cu[1:] - cu[:-1])  # the first new position of each sequence
    pos = first[b] + i - cu[b]
    at, blk = table[b, pos // page], pos % page // block
    fat = table.gather(1, (first // page)[:, None])[:, 0]
    fblk, old = first % page // block, first % block  # its block, and the old rows there
    keep = torch.arange(block, device=cu.device) < old[:, None]  # [B, block]
    out = {}
    for n in "kv":
        x = s[n].float() if s["packed"] else s[n].float().transpose(0, 1).flatten(1, 2)
        x = x.transpose(0, 1)  # [rows, Hk, d]
        P, Hk, _, d = s[n + "_cache"].shape
        codes = s[n + "_cache"].view(P, Hk, nb, block, d)
        scale = s[n + "_scale"]
        fine = torch.isfinite(x)
        amax = torch.where(fine, x, 0.0).abs().amax(-1)
        most = torch.zeros(P * nb, Hk, device=x.device).scatter_reduce_(
            0, (at * nb + blk)[:, None].expand(-1, Hk), amax, "amax").view(P, nb, Hk)
        was, kept = scale[fat, :, fblk], codes[fat, :, fblk].float()  # of the blocks added to
        scale[at, :, blk] = _power(most[at, blk])
        now = scale[fat, :, fblk]
        now = torch.where((old > 0)[:, None], torch.maximum(now, was), now)
        scale[fat, :, fblk] = now
        again = _codes(kept * (was / now)[..., None, None])
        raw = codes.view(torch.uint8)
        raw[fat, :, fblk] = torch.where(keep[:, None, :, None], again.view(torch.uint8),
                                        raw[fat, :, fblk])
        y = torch.where(fine, x / scale[at, :, blk][..., None], torch.nan)
        raw[at, :, blk, pos % block] = _codes(y).view(torch.uint8)
        out[n], out[n + "_scale"] = s[n + "_cache"], scale
    return out


def _plain_read(s):
    c = s["case"]
    cu, page = s["cu"].long(), c["page"]
    i = torch.arange(s["total"], device=cu.device)
    b = torch.searchsorted(cu, i, right=True) - 1
    pos = i - cu[b]
    at, slot = s["table"].long()[b, pos // page], pos % page
    out = {}
    for n in "kv":
        x = s[n + "_cache"].view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn)
        x = x.float() * s[n + "_scale"][at, :, slot // c["block"]][..., None]
        out[n] = x.bfloat16().transpose(0, 1).contiguous()
    return out


def _own(s):
    import flash_attention_gb300 as fa

    c = s["case"]
    cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if c["op"] == "attend":
        o, lse = fa.q8_paged_attention(s["q"], *cache, s["table"], s["lengths"],
                                       scale=s["scale"], causal=c["causal"])
        return {"o": o, "lse": lse}
    if c["op"] == "write":
        fa.q8_cache_write(s["k"], s["v"], *cache, s["table"], s["lengths"],
                          cu_seqlens=s["cu"] if s["packed"] else None)
        return {"k": cache[0], "v": cache[1], "k_scale": cache[2], "v_scale": cache[3]}
    k, v = fa.q8_cache_read(*cache, s["table"], s["cu"], s["total"])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read}[
        state["case"]["op"]](state)


# ------------------------------------------------------------- the definitions, in 64 bits
def _e4m3(y):
    """y rounded to e4m3 (ties to even), in 64 bits: steps of 2^(e - 3) in the binade of 2^e, and
    of 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _logical(s, n, b, pos):
    """(codes [rows, Hk, d], scales [rows, Hk]) at the positions `pos` of sequence b."""
    page, block = s["case"]["page"], s["case"]["block"]
    at, slot = s["table"][b].long()[pos // page], pos % page
    codes = s[n + "_cache"].view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn)
    return codes.double(), s[n + "_scale"][at, :, slot // block].double()


def _exact_attend(s):
    c, q = s["case"], s["q"].double()
    B, H, lq, d = q.shape
    Hk = c["Hk"]
    o = torch.zeros(B, H, lq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, lq), -torch.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lengths"].tolist()):
        j = torch.arange(n, device=q.device)
        (k, ks), (v, vs) = _logical(s, "k", b, j), _logical(s, "v", b, j)
        i = torch.arange(lq, device=q.device)[:, None]
        a = torch.einsum("hgid,jhd->hgij", q[b].view(Hk, H // Hk, lq, d), k * ks[..., None])
        a = a * s["scale"]
        if c["causal"]:
            a = torch.where(j <= n - lq + i, a, -torch.inf)
        z = torch.logsumexp(a, -1)
        w = torch.exp(a - z.clamp(min=-1e300)[..., None])
        o[b] = torch.einsum("hgij,jhd->hgid", w, v * vs[..., None]).view(H, lq, d)
        lse[b] = z.view(H, lq)
    return {"o": o, "lse": lse}


def _exact_write(s):
    c = s["case"]
    page, block, cu = c["page"], c["block"], s["cu"].tolist()
    out = {}
    for n in "kv":
        codes, scale = s[n + "_cache"].double(), s[n + "_scale"].double()
        for b, length in enumerate(s["lengths"].tolist()):
            x = s[n][:, cu[b]:cu[b + 1]] if s["packed"] else s[n][b]  # [Hk, rows, d]
            first = length - x.shape[1]
            start = first // block * block  # from the start of the block that is added to
            rows = -(-length // block) * block - start
            new = torch.zeros(x.shape[0], rows, x.shape[2], dtype=torch.float64, device=x.device)
            new[:, first - start:length - start] = x.double()
            fine = torch.isfinite(new)
            amax = torch.where(fine, new, 0.0).abs().view(x.shape[0], -1, block, x.shape[2])
            amax = amax.amax((2, 3)).clamp(min=448 * 2.0 ** -100)
            power = torch.exp2(torch.round(torch.log2(amax / 448)))  # [Hk, blocks]
            power = torch.where(448 * power < amax, 2 * power, power)
            pos = torch.arange(start, length, device=x.device)
            kept, was = _logical(s, n, b, pos)
            if first > start:
                power[:, 0] = torch.maximum(power[:, 0], was[0])
            each = power.repeat_interleave(block, 1)[:, :length - start].T  # [rows, Hk]
            y = torch.where(fine, new, torch.nan).transpose(0, 1)[:length - start]
            y = torch.where((pos < first)[:, None, None], kept * (was / each)[..., None],
                            y / each[..., None])
            at = s["table"][b].long()[pos // page]
            codes[at, :, pos % page] = _e4m3(y)
            scale[at, :, pos % page // block] = each
        out[n], out[n + "_scale"] = codes, scale
    return out


def _exact_read(s):
    lens, out = (s["cu"][1:] - s["cu"][:-1]).tolist(), {}
    for n in "kv":
        rows = []
        for b, length in enumerate(lens):
            codes, scale = _logical(s, n, b, torch.arange(length, device="cuda"))
            rows.append(codes * scale[..., None])
        out[n] = torch.cat(rows).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "write": _exact_write, "read": _exact_read}[case["op"]](s)
