"""The operators of a step that decodes drafted tokens, as work to be measured: rotating queries and
keys by their positions (with its gradient), appending keys and values to a paged cache with the
rotation on the way, attention for a tree of drafted tokens over that cache, and keeping the rows of
the accepted ones.

The cache holds bf16 keys and values in pages, [num_pages, kv_heads, page, dim]. Key j of a sequence
is in page table[b, j // page], slot j % page.

  rotate: with the angle a = position * inv_freq[i] (inv_freq in 64 bits), each pair (x1, x2) of the
          first 2 * len(inv_freq) elements of a row becomes
          mscale * (x1 cos a - x2 sin a, x1 sin a + x2 cos a); the others stay. Pairs are elements
          i and i + len(inv_freq), or 2 i and 2 i + 1 (interleaved). The gradient turns back by the
          same angle.
  append: the n new rows of sequence b become its positions length - n .. length - 1, keys rotated
          and values as they are; the queries of the same rows come back rotated
  attend: o = softmax(scale * q k^T) v and the natural logarithm of the softmax's sum for the T
          nodes of a tree, a sequence's last T keys: a node sees every key before them, and of them
          those that its row of the mask names
  keep:   of a sequence's last T keys the count[b] that keep[b] names (ascending) move to the front
          of the T; the length becomes length - T + count

`run` computes them in elementary operations, or with `own` set through the framework's calls.
"""
import math
import random

import torch

own = False

SPARE = 5  # pages of a cache that no sequence uses


def _attend(name, B, H, Hk, d, T, page, lo, hi, lens, shared=False):
    return dict(name=name, op="attend", B=B, H=H, Hk=Hk, d=d, T=T, page=page, min_len=lo,
                max_len=hi, lens=lens, shared=shared)


def _append(name, B, H, Hk, d, rot, page, past, lo, hi, lens, inter=False, tree=False, far=0):
    return dict(name=name, op="append", B=B, H=H, Hk=Hk, d=d, rot=rot, page=page, past=past,
                min_len=lo, max_len=hi, lens=lens, inter=inter, tree=tree, far=far)


def _rotate(name, B, H, Hk, n, d, rot, layout, inter, back, far=0, mscale=1.0):
    return dict(name=name, op="rotate", B=B, H=H, Hk=Hk, n=n, d=d, rot=rot, layout=layout,
                inter=inter, back=back, far=far, mscale=mscale)


def _keep(name, B, Hk, d, T, M, page, past, lens):
    return dict(name=name, op="keep", B=B, Hk=Hk, d=d, T=T, M=M, page=page, past=past, lens=lens)


def listed():
    return [
        # a small tree behind one short conversation: the latency of a call
        _attend("tree of 8, 1x37", 1, 4, 4, 128, 8, 16, 37, 37, 1),
        # a server's batch, grouped heads, small pages, a tree of its own for each sequence
        _attend("tree of 32, 16x16k", 16, 32, 8, 128, 32, 16, 2048, 16384, 2),
        # many short conversations, every head its own keys, one odd tree for all
        _attend("tree of 17, 100x2k d64", 100, 8, 8, 64, 17, 64, 17, 2047, 3, shared=True),
        # wide heads, odd lengths, as many rows a kv head as the arithmetic counts for something
        _attend("tree of 64, 7x8k d256", 7, 16, 4, 256, 64, 32, 501, 8191, 4),
        # the largest batch, a narrow tree
        _attend("tree of 12, 64x16k", 64, 32, 8, 128, 12, 32, 1024, 16384, 5, shared=True),
        # the token that each sequence of a decoding batch adds
        _append("append 16x1", 16, 32, 8, 128, 128, 16, 16383, 1, 1, 6),
        # a drafted tree for each of many sequences, far positions, a quarter of the head rotated
        _append("append 100x33 d64", 100, 8, 8, 64, 16, 64, 500, 33, 33, 7, inter=True, tree=True,
                far=1000000),
        # a batch of prompts of mixed lengths
        _append("append 16x8k", 16, 32, 8, 128, 128, 16, 0, 256, 8192, 8),
        # a training step's queries and keys on their way to attention, out of their projections
        _rotate("rotate 2x4096", 2, 32, 8, 4096, 128, 128, "rows", False, False),
        # the gradients' way back: packed sequences, half of wide heads, stretched positions
        _rotate("rotate back 8k d256", 5, 16, 4, 8191, 256, 128, "packed", True, True, mscale=1.25),
        # one sequence's accepted path
        _keep("keep 1", 1, 8, 128, 16, 4, 16, 1000, 9),
        # a large batch's accepted paths
        _keep("keep 64", 64, 8, 128, 64, 24, 16, 16000, 10),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("attend", "attend", "append", "rotate", "keep"))
    d = rng.choice((64, 128, 256))
    Hk, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((8, 16, 32, 64, 128))
    rot = rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= d])
    lens, inter = rng.randrange(1 << 20), rng.random() < 0.5
    if op == "rotate":
        B = log(1, 16)
        n = log(1, max(2, min(8192, (1 << 25) // (B * Hk * (1 + G) * d))))
        return dict(op=op, B=B, H=G * Hk, Hk=Hk, n=n, d=d, rot=rot,
                    layout=rng.choice(("heads", "rows", "packed")), inter=inter,
                    back=rng.random() < 0.5, far=rng.choice((0, 0, 5000, 2000000)),
                    mscale=rng.choice((1.0, 1.2)))
    if op == "keep":
        T = log(2, 200)
        return dict(op=op, B=log(1, 96), Hk=Hk, d=d, T=T, M=rng.randint(1, min(T, 40)), page=page,
                    past=rng.choice((0, 50, 3000)), lens=lens)
    B = log(1, 96)
    cost = (1 << 29) if op == "attend" else (1 << 28) // (2 + G)
    most = max(64, min(16384, cost // (B * Hk * d)))
    hi = log(8, most)
    lo = max(1, hi // rng.choice((1, 2, 30)))
    if op == "attend":
        T = log(1, 128)
        while T > 1 and B * G * Hk * T * (hi + T) * d > 1 << 34:
            T = T // 2 + T % 2
        return dict(op=op, B=B, H=G * Hk, Hk=Hk, d=d, T=T, page=page, min_len=lo + T - 1,
                    max_len=hi + T - 1, lens=lens, shared=rng.random() < 0.4)
    kind = rng.random()
    hi = 1 if kind < 0.3 else log(2, 100) if kind < 0.6 else min(hi, 8192)
    lo = 1 if hi == 1 else hi if kind < 0.6 else min(lo, hi)
    return dict(op=op, B=B, H=G * Hk, Hk=Hk, d=d, rot=rot, page=page,
                past=rng.choice((0, 9, 700)), min_len=lo, max_len=hi, lens=lens, inter=inter,
                tree=kind < 0.6 and rng.random() < 0.5, far=rng.choice((0, 0, 2000000)))


def _lengths(case):
    """(new or cached rows of each sequence, rows that were there before); the last sequence is
    the longest."""
    r = random.Random(case["lens"])
    if case["op"] == "keep":
        return [case["T"]] * case["B"], [r.randint(0, case["past"]) for _ in range(case["B"])]
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["B"])]
    lens[-1] = case["max_len"]
    past = [r.randint(0, case["past"]) if case["op"] == "append" else 0 for _ in lens]
    return lens, past


def _counts(case):
    r = random.Random(case["lens"] + 1)
    return [r.randint(min(1, case["M"]), case["M"]) for _ in range(case["B"])]


def _packed_lengths(case):
    """Rows of each sequence of a packed rotation; the first is the longest."""
    r = random.Random(case["n"])
    return [case["n"]] + [r.randint(0, case["n"]) for _ in range(case["B"] - 1)]


def work(case):
    Hk, d = case["Hk"], case["d"]
    if case["op"] == "rotate":
        rows = sum(_packed_lengths(case)) if case["layout"] == "packed" else case["B"] * case["n"]
        x = rows * (case["H"] + Hk)
        return {"bytes": 4 * x * d, "flops": 3 * x * case["rot"]}
    if case["op"] == "keep":
        return {"bytes": sum(_counts(case)) * Hk * d * 8, "flops": 0}
    rows = sum(_lengths(case)[0])
    table = 4 * sum(-(-n // case["page"]) for n in _lengths(case)[0])
    if case["op"] == "append":
        return {"bytes": 4 * rows * d * (2 * Hk + case["H"]) + table,
                "flops": 3 * rows * case["rot"] * (Hk + case["H"])}
    q = case["B"] * case["H"] * case["T"]
    mask = case["T"] ** 2 * (1 if case["shared"] else case["B"])
    return {"bytes": 4 * rows * Hk * d + table + q * (4 * d + 4) + mask,
            "flops": 4 * d * case["H"] * case["T"] * rows}


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _trees(g, B, T):
    """(ancestors and itself of each node [B, T, T], its depth) of random trees: a node's parent is
    one of the few nodes before it, or the sequence itself."""
    back = torch.randint(1, 6, (B, T), generator=g, device="cuda")
    parent = torch.arange(T, device="cuda") - back
    sees = torch.eye(T, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    b = torch.arange(B, device="cuda")
    for i in range(1, T):
        up = parent[:, i]
        sees[:, i] |= sees[b, up.clamp(min=0)] & (up >= 0)[:, None]
    return sees, sees.sum(-1) - 1


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hk, d = case["B"], case["Hk"], case["d"]
    s = dict(case=case)
    if "rot" in case:
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                                  -2 * i / case["rot"])
    if case["op"] == "rotate":
        H, n = case["H"], case["n"]
        if case["layout"] == "packed":
            s["cu"] = _ints(_offsets(_packed_lengths(case)))
            s["total"] = sum(_packed_lengths(case))
            s["q"], s["k"] = _bf16(g, H, s["total"], d), _bf16(g, Hk, s["total"], d)
        elif case["layout"] == "rows":  # columns of one projection's output
            wide = _bf16(g, B, n, (H + 2 * Hk) * d).unflatten(2, (H + 2 * Hk, d)).transpose(1, 2)
            s["q"], s["k"] = wide[:, :H], wide[:, H:H + Hk]
        else:
            s["q"], s["k"] = _bf16(g, B, H, n, d), _bf16(g, B, Hk, n, d)
        s["offset"] = case["far"]
        return s
    page = case["page"]
    lens, past = _lengths(case)
    total = [n + p for n, p in zip(lens, past)]
    per = -(-max(total) // page)
    pages = B * per + SPARE
    s["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(B, per).int()
    s["lengths"] = _ints(total)
    # keys with a few large channels
    large = 1 + 3 * (torch.rand(Hk, 1, d, generator=g, device="cuda") < 0.03)
    s["k_cache"] = (_bf16(g, pages, Hk, page, d) * large).bfloat16()
    s["v_cache"] = _bf16(g, pages, Hk, page, d)
    if case["op"] == "attend":
        s["q"], s["scale"] = _bf16(g, B, case["H"], case["T"], d), d ** -0.5
        sees, _ = _trees(g, 1 if case["shared"] else B, case["T"])
        s["mask"] = sees[0].contiguous() if case["shared"] else sees
    elif case["op"] == "append":
        H = case["H"]
        s["packed"] = case["min_len"] != case["max_len"] or case["max_len"] > 100
        s["total"], s["cu"] = sum(lens), _ints(_offsets(lens))
        n = s["total"] if s["packed"] else case["max_len"]
        wide = _bf16(g, 1 if s["packed"] else B, n, (H + 2 * Hk) * d)
        wide = wide.unflatten(2, (H + 2 * Hk, d)).transpose(1, 2)  # one projection's output
        wide = wide[0] if s["packed"] else wide
        at = wide.dim() - 3
        s["q"], s["k"], s["v"] = (wide.narrow(at, 0, H), wide.narrow(at, H, Hk),
                                  wide.narrow(at, H + Hk, Hk))
        # positions that are not those of the cache: a tree's depths, a conversation cut in front
        s["positions"] = None
        if case["tree"] or case["far"]:
            ahead = torch.arange(n, device="cuda").repeat(B, 1)
            if case["tree"]:
                ahead = _trees(g, B, n)[1]
            first = s["lengths"].long() - torch.tensor(lens, device="cuda") + case["far"]
            if s["packed"]:
                ahead = torch.cat([torch.arange(m, device="cuda") for m in lens])
                first = torch.repeat_interleave(first, torch.tensor(lens, device="cuda"))
                s["positions"] = (first + ahead).int()
            else:
                s["positions"] = (first[:, None] + ahead).int()
    else:
        T, M = case["T"], case["M"]
        s["counts"] = _ints(_counts(case))
        # a path: ascending nodes (those behind the count are any)
        s["keep"] = torch.rand(B, T, generator=g, device="cuda").topk(M).indices.sort().values.int()
    return s


# --------------------------------------------------------------------- the plain forms
def _turn(x, angle, mscale, inter):
    """The rotation of x [..., rows, d] by angle [..., rows, rot / 2] (64 bits), in 32 bits."""
    rot = 2 * angle.shape[-1]
    cos, sin = (mscale * angle.cos()).float(), (mscale * angle.sin()).float()
    y = x.float()
    if inter:
        x1, x2 = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1).flatten(-2)
    else:
        x1, x2 = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
    return torch.cat((turned, y[..., rot:]), -1).bfloat16()


def _plain_rotate(s):
    c = s["case"]
    if c["layout"] == "packed":
        i = torch.arange(s["total"], device="cuda")
        cu = s["cu"].long()
        pos = i - cu[torch.searchsorted(cu, i, right=True) - 1]
    else:
        pos = torch.arange(c["n"], device="cuda")
    angle = (pos + s["offset"]).double()[:, None] * s["inv_freq"]
    if c["back"]:
        angle = -angle
    return {n: _turn(s[n], angle, c["mscale"], c["inter"]) for n in "qk"}


def _plain_append(s):
    c = s["case"]
    cu, length, page = s["cu"].long(), s["lengths"].long(), c["page"]
    i = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    pos = length[b] - (cu[1:] - cu[:-1])[b] + i - cu[b]
    at = s["table"].long()[b, pos // page]
    turn = pos if s["positions"] is None else s["positions"].reshape(-1)
    angle = turn.double()[:, None] * s["inv_freq"]
    if not s["packed"]:
        angle = angle.view(c["B"], 1, c["max_len"], -1)
    k, q = (_turn(s[n], angle, 1.0, c["inter"]) for n in "kq")
    for x, cache in ((k, s["k_cache"]), (s["v"], s["v_cache"])):
        rows = x.transpose(0, 1) if s["packed"] else x.transpose(1, 2).flatten(0, 1)
        cache[at, :, pos % page] = rows
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _plain_attend(s):
    c, q, table = s["case"], s["q"], s["table"].long()
    B, H, T, d = q.shape
    Hk = c["Hk"]

    def gathered(n):  # [B, pages, Hk, page, d] -> [B, Hk, keys, d]
        return s[n][table].transpose(1, 2).reshape(B, Hk, -1, d).float()

    k, v = gathered("k_cache"), gathered("v_cache")
    a = torch.matmul(q.float().view(B, Hk, -1, d), k.transpose(2, 3)) * s["scale"]
    keys = a.shape[-1]
    node = torch.arange(keys, device="cuda") - (s["lengths"].long()[:, None] - T)  # [B, keys]
    named = s["mask"].expand(B, T, T).gather(2, node.clamp(0, T - 1)[:, None].expand(B, T, keys))
    seen = ((node < 0)[:, None] | named) & (node < T)[:, None]  # [B, T, keys]
    a = a.view(B, Hk, H // Hk, T, keys).masked_fill_(~seen[:, None, None], -torch.inf)
    top = a.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(a - top)
    z = p.sum(-1, keepdim=True)
    v = torch.where((node < T)[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, Hk, -1, keys), v).view(B, Hk, -1, T, d)
    o = torch.where(z > 0, o / z, 0.0)
    return {"o": o.reshape(B, H, T, d).bfloat16(), "lse": (top + z.log()).reshape(B, H, T)}


def _plain_keep(s):
    c = s["case"]
    page, table, count = c["page"], s["table"].long(), s["counts"].long()
    base = s["lengths"].long() - c["T"]
    b, i = torch.nonzero(torch.arange(c["M"], device="cuda") < count[:, None], as_tuple=True)
    src, dst = base[b] + s["keep"].long()[b, i], base[b] + i
    for n in ("k_cache", "v_cache"):
        rows = s[n][table[b, src // page], :, src % page]
        s[n][table[b, dst // page], :, dst % page] = rows
    return {"k": s["k_cache"], "v": s["v_cache"], "lengths": (base + count).int()}


def _own(s):
    import flash_attention_gb300 as fa

    c = s["case"]
    if c["op"] == "rotate":
        call = fa.rotary_bwd if c["back"] else fa.rotary_fwd
        q, k = call(s["q"], s["k"], s["inv_freq"], offset=s["offset"], scale=c["mscale"],
                    interleaved=c["inter"], cu_seqlens=s.get("cu"))
        return {"q": q, "k": k}
    cache = s["k_cache"], s["v_cache"]
    if c["op"] == "append":
        q = fa.paged_cache_append(s["k"], s["v"], *cache, s["table"], s["lengths"], q=s["q"],
                                  inv_freq=s["inv_freq"], positions=s["positions"],
                                  interleaved=c["inter"],
                                  cu_seqlens=s["cu"] if s["packed"] else None)
        return {"q": q, "k": cache[0], "v": cache[1]}
    if c["op"] == "keep":
        lengths = fa.paged_cache_keep(*cache, s["table"], s["lengths"], s["keep"], s["counts"],
                                      c["T"])
        return {"k": cache[0], "v": cache[1], "lengths": lengths}
    o, lse = fa.paged_tree_attention(s["q"], *cache, s["table"], s["lengths"], s["mask"],
                                     scale=s["scale"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "append": _plain_append, "rotate": _plain_rotate,
            "keep": _plain_keep}[state["case"]["op"]](state)


# ------------------------------------------------------------- the definitions, in 64 bits
def _exact_turn(x, pos, c):
    """x [heads, rows, d] turned by its rows' positions, as complex numbers."""
    half, x = c["rot"] // 2, x.double()
    angle = torch.stack([pos.double() * 10000.0 ** (-i / half) for i in range(half)], -1)
    angle = -angle if c.get("back") else angle
    head = x[..., :2 * half]
    head = head.unflatten(-1, (half, 2)) if c["inter"] else head.unflatten(-1, (2, half)).mT
    z = torch.view_as_complex(head.contiguous())
    z = z * torch.polar(torch.full_like(angle, c.get("mscale", 1.0)), angle)
    pair = torch.view_as_real(z)
    out = x.clone()
    out[..., :2 * half] = (pair if c["inter"] else pair.mT).flatten(-2)
    return out


def _exact_rotate(s):
    c, out = s["case"], {}
    for n in "qk":
        if c["layout"] == "packed":
            pos = torch.cat([torch.arange(m, device="cuda") for m in _packed_lengths(c)])
            out[n] = _exact_turn(s[n], pos + c["far"], c)
        else:
            pos = torch.arange(c["n"], device="cuda") + c["far"]
            out[n] = torch.stack([_exact_turn(x, pos, c) for x in s[n]])
    return out


def _exact_append(s):
    c = s["case"]
    cu, page = s["cu"].tolist(), c["page"]
    q, out = [], {"k": s["k_cache"].double(), "v": s["v_cache"].double()}
    for b, length in enumerate(s["lengths"].tolist()):
        new = {n: s[n][:, cu[b]:cu[b + 1]] if s["packed"] else s[n][b] for n in "qkv"}
        pos = torch.arange(length - new["k"].shape[1], length, device="cuda")
        turn = pos
        if s["positions"] is not None:
            turn = s["positions"][cu[b]:cu[b + 1]] if s["packed"] else s["positions"][b]
        at = s["table"][b].long()[pos // page]
        out["k"][at, :, pos % page] = _exact_turn(new["k"], turn, c).transpose(0, 1)
        out["v"][at, :, pos % page] = new["v"].double().transpose(0, 1)
        q.append(_exact_turn(new["q"], turn, c))
    out["q"] = torch.cat(q, 1) if s["packed"] else torch.stack(q)
    return out


def _exact_attend(s):
    c, q = s["case"], s["q"].double()
    B, H, T, d = q.shape
    Hk, page = c["Hk"], c["page"]
    o = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        j = torch.arange(n, device="cuda")
        at = s["table"][b].long()[j // page]
        k, v = (s[x][at, :, j % page].double() for x in ("k_cache", "v_cache"))  # [keys, Hk, d]
        mask = s["mask"] if c["shared"] else s["mask"][b]
        sees = torch.ones(T, n, dtype=torch.bool, device="cuda")
        sees[:, max(0, n - T):] = mask[:, max(0, T - n):]
        for h in range(H):
            a = torch.where(sees, q[b, h] @ k[:, h // (H // Hk)].T * s["scale"], -math.inf)
            lse[b, h] = torch.logsumexp(a, -1)
            w = torch.exp(a - lse[b, h].clamp(min=-1e300)[:, None])
            o[b, h] = w @ v[:, h // (H // Hk)]
    return {"o": o, "lse": lse}


def _exact_keep(s):
    page, T, out = s["case"]["page"], s["case"]["T"], {}
    counts = s["counts"].tolist()
    for n in ("k", "v"):
        x = s[n + "_cache"].double()
        for b, length in enumerate(s["lengths"].tolist()):
            row = s["table"][b].long()
            pos = torch.arange(length - T, length, device="cuda")
            tree = x[row[pos // page], :, pos % page]
            to = pos[:counts[b]]
            x[row[to // page], :, to % page] = tree[s["keep"][b, :counts[b]].long()]
        out[n] = x
    lengths = [m - T + n for m, n in zip(s["lengths"].tolist(), counts)]
    return {**out, "lengths": _ints(lengths)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "rotate": _exact_rotate,
            "keep": _exact_keep}[case["op"]](s)
