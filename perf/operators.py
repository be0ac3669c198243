"""The quantised key-value cache: what is measured of it, and its plain form.

Three operators: tokens are quantised as they are written into a paged cache, rows of the cache are read back as
bf16, and new tokens attend to the cache.  The cache is a uint8 tensor [pages, heads, page_size, token_bytes], in which
a page of one head is a run of 16-token tiles, each

    16 rows of K codes (D * bits / 8 bytes) | 16 rows of V codes | 16 rows of (scale, bias) fp16 pairs,

a row's pairs being those of its K groups and then of its V groups.  Codes are packed LSB first.
"""
import math

import numpy as np
import torch

own = False

TILE = 16  # tokens of a tile


def listed():
    return [
        # one chat turn, just begun: latency is all there is
        attend("attend one, short", batch=1, shortest=211, longest=211),
        # one user with a long document
        attend("attend one, long", batch=1, shortest=65521, longest=65521, page=64),
        # a serving batch, requests at every stage
        attend("attend batch, ragged", batch=64, shortest=1, longest=8192),
        # a larger model's heads with 8-bit codes, long contexts
        attend("attend batch, 8 bits", batch=32, shortest=4096, longest=16384, q_heads=64, G=128, bits=8, page=32),
        # five drafted tokens a sequence, verified at once
        attend("attend drafted tokens", batch=16, tokens=5, shortest=100, longest=3001, G=32),
        # a layer with a sliding window and a KV head for each query head
        attend("attend window", batch=48, shortest=1, longest=6000, q_heads=16, heads=16, D=64, bits=8, page=64, window=1000),
        # wide heads, few of them
        attend("attend wide heads", batch=24, shortest=1999, longest=5001, q_heads=16, heads=2, D=256, page=128),
        # the decode step's own write: a token for each sequence
        write("write one token", batch=64, shortest=1, longest=4000, each=1),
        # prompts of a prefill batch, one after the other
        write("write prompts", batch=9, shortest=17, longest=2011, each=0),
        # a chunk of one long prompt behind what is cached of it, 8-bit codes
        write("write a chunk, 8 bits", batch=1, shortest=9001, longest=9001, each=4096, G=128, bits=8, page=64),
        # a short shared prefix, read for the prefill that follows it
        read("read a prefix", batch=1, shortest=129, longest=129, G=32, bits=8),
        # whole contexts, read back when requests move to another form of attention
        read("read contexts", batch=16, shortest=2048, longest=14001, page=32),
    ]


def attend(name, batch, shortest, longest, tokens=1, q_heads=32, heads=8, D=128, G=64, bits=4, page=16, window=0):
    return dict(name=name, op="attend", batch=batch, shortest=shortest, longest=longest, tokens=tokens, q_heads=q_heads, heads=heads, D=D, G=G, bits=bits, page=page, window=window)


def write(name, batch, shortest, longest, each, heads=8, D=128, G=64, bits=4, page=16):
    """`each` new tokens a sequence; 0: all of its tokens are new."""
    return dict(name=name, op="write", batch=batch, shortest=shortest, longest=longest, each=each, heads=heads, D=D, G=G, bits=bits, page=page)


def read(name, batch, shortest, longest, heads=8, D=128, G=64, bits=4, page=16):
    """All tokens of every sequence."""
    return dict(name=name, op="read", batch=batch, shortest=shortest, longest=longest, heads=heads, D=D, G=G, bits=bits, page=page)


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    D = rng.choice((64, 128, 128, 256))
    form = dict(D=D, G=rng.choice([g for g in (32, 64, 128) if g <= D]), bits=rng.choice((4, 4, 8)), page=rng.choice((16, 32, 64, 128, 256)))
    op = rng.choice(("attend", "attend", "attend", "write", "read"))
    batch = spread(1, 96)
    # so many cached values of K at most in all, with every sequence at its longest
    most = 270_000_000 if op == "attend" else 100_000_000
    heads = rng.choice((1, 2, 4, 8, 8, 16))
    longest = spread(1, max(2, min(100_000, most // (batch * heads * D))))
    shortest = rng.randint(max(1, longest // 20), longest)
    case = dict(op=op, batch=batch, shortest=shortest, longest=longest, heads=heads, **form)
    if op == "attend":
        case |= dict(tokens=rng.choice((1, 1, 1, 2, 3, 6)), q_heads=heads * rng.choice((1, 2, 4, 7, 8, 16)), window=rng.choice((0, 0, spread(16, 4096))))
    if op == "write":
        case |= dict(each=rng.choice((0, 1, 1, min(shortest, spread(2, 600)))))
    return case


def lengths(case):
    """The sequences' lengths: they belong to the case, not to the seed, so that its work is the same for every seed."""
    n = np.random.RandomState(case["longest"] + 7 * case["batch"]).randint(case["shortest"], case["longest"] + 1, case["batch"])
    n[0] = case["longest"]
    return n


def row_bytes(case):
    return case["D"] * case["bits"] // 8


def token_bytes(case):
    return 2 * row_bytes(case) + 8 * case["D"] // case["G"]


def news(case):
    """New (or read) tokens of each sequence."""
    n = lengths(case)
    return n if case["op"] == "read" or not case["each"] else np.minimum(n, case["each"])


def work(case):
    H, D, n = case["heads"], case["D"], lengths(case)
    if case["op"] == "attend":
        rows = case["batch"] * case["tokens"] * case["q_heads"]
        # what the sequence's new tokens see between them: the last one's position down to the first one's window
        seen = np.minimum(n, case["window"] + case["tokens"] - 1) if case["window"] else n
        total = int(seen.sum())
        return {"bytes": total * H * token_bytes(case) + 4 * rows * D, "flops": 4 * total * case["tokens"] * case["q_heads"] * D}
    total = int(news(case).sum())
    values = total * H * D * 2
    moved = 2 * values + total * H * token_bytes(case)
    # a write's pass also reads its own rows back
    return {"bytes": moved * (2 if case["op"] == "write" else 1), "flops": values * (8 if case["op"] == "write" else 2)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, D, page = case["batch"], case["heads"], case["D"], case["page"]
    n = torch.from_numpy(lengths(case)).cuda()
    width = -(-case["longest"] // page)
    pages = B * width + 3
    cache = torch.zeros(pages, H, page, token_bytes(case), dtype=torch.uint8, device="cuda")
    table = torch.randperm(pages, generator=g, device="cuda")[: B * width].view(B, width)
    # keys have channels that lie off zero, values do not
    shape = (pages * page // TILE, TILE, H, D)
    off = torch.randn(H, D, generator=g, device="cuda").pow(3).div(4).clamp(-4, 4)
    k = torch.randn(shape, generator=g, device="cuda").add_(off).bfloat16()
    v = torch.randn(shape, generator=g, device="cuda").mul_(0.7).bfloat16()
    kq, vq = quantise(k, case), quantise(v, case)
    del k, v
    tile = torch.cat((kq[0].transpose(1, 2).flatten(2), vq[0].transpose(1, 2).flatten(2), torch.cat((kq[1], vq[1]), -1).transpose(1, 2).flatten(2)), -1)  # [tiles, H, bytes]
    cache.view(pages, H, page // TILE, -1).copy_(tile.view(pages, page // TILE, H, -1).transpose(1, 2))
    del kq, vq, tile
    # what lies behind a sequence's end was never written: anything may stand there, NaN for scales too
    behind = torch.arange(width * page, device="cuda")[None] >= n[:, None]
    at = place(table.repeat_interleave(page, 1)[behind], torch.arange(width * page, device="cuda").expand(B, -1)[behind], page)
    cells(cache, case)[2].movedim(1, 3)[at] = 255
    state = dict(case=case, cache=cache, table=table.int().contiguous(), lens=n.int())
    if case["op"] == "attend":
        state["q"] = torch.randn(B, case["tokens"], case["q_heads"], D, generator=g, device="cuda").mul_(1.5).bfloat16()
        return state
    new = news(case)
    state["offsets"] = torch.from_numpy(np.concatenate(([0], new.cumsum())).astype(np.int32)).cuda()
    state["rows"] = int(new.sum())
    if case["op"] == "write":
        # keys and values lie in one projection's output, as a layer gives them
        kv = torch.randn(state["rows"], 2, H, D, generator=g, device="cuda")
        kv[:, 0] += off
        state["k"], state["v"] = kv.bfloat16().unbind(1)
    return state


def run(state):
    case = state["case"]
    cache, table, lens = state["cache"], state["table"], state["lens"]
    if own:
        import weight_only_group_b200 as aq

        if case["op"] == "attend":
            return aq.aq_kv_attention(state["q"], cache, table, lens, case["G"], case["bits"], window=case["window"])
        if case["op"] == "write":
            aq.aq_kv_append(cache, state["k"], state["v"], table, lens, case["G"], case["bits"], offsets=state["offsets"])
        return aq.aq_kv_read(cache, table, lens, state["rows"], case["D"], case["G"], case["bits"], offsets=state["offsets"])
    if case["op"] == "attend":
        return plain_attention(state["q"], cache, table, lens, case)
    seq, pos = rows_at(state["offsets"], lens, state["rows"])
    at = place(table.long()[seq, pos // case["page"]], pos, case["page"])
    if case["op"] == "write":
        plain_write(cache, state["k"], state["v"], at, case)
    return plain_read(cache, at, case)


# The plain form


def cells(cache, case):
    """Views of the cache: K codes, V codes [pages, heads, tiles, 16, bytes of a row], and pairs [.., 16, bytes of a row's pairs]."""
    rb = row_bytes(case)
    tiles = cache.flatten(2).unflatten(2, (-1, TILE * token_bytes(case)))
    return tuple(tiles[..., a:b].unflatten(3, (TILE, -1)) for a, b in ((0, TILE * rb), (TILE * rb, 2 * TILE * rb), (2 * TILE * rb, None)))


def place(page_id, pos, page):
    """(page, tile, row) of positions."""
    return page_id.long(), pos % page // TILE, pos % TILE


def rows_at(offsets, lens, rows):
    """The sequence and the position of each row: a sequence's rows are its last tokens."""
    r = torch.arange(rows, device=offsets.device)
    seq = torch.searchsorted(offsets.long(), r, right=True) - 1
    return seq, lens.long()[seq] - offsets.long()[seq + 1] + r


def quantise(x, case):
    """x [.., D] -> codes as bytes [.., D * bits / 8] and (scale, bias) pairs as bytes [.., 4 * groups]."""
    top = 2 ** case["bits"] - 1
    x = x.float().unflatten(-1, (-1, case["G"]))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    # (a tensor divisor: a division by a plain number is a product with its rounded reciprocal)
    scale = ((high - low) / torch.full_like(low, top)).half()
    bias = low.half()
    q = ((x - bias.float()) / scale.float()).round().clamp(0, top)
    q = torch.where(scale == 0, torch.zeros_like(q), q).to(torch.uint8).flatten(-2)
    if case["bits"] == 4:
        q = q[..., 0::2] | q[..., 1::2] << 4
    return q, torch.cat((scale, bias), -1).flatten(-2).view(torch.uint8)


def values(codes, pairs, case):
    """What codes [.., bytes] and pairs [.., bytes] stand for, in 32 bits [.., D]."""
    if case["bits"] == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    pairs = pairs.contiguous().view(torch.float16).float().unflatten(-1, (-1, 2))
    return (codes.float().unflatten(-1, (-1, case["G"])) * pairs[..., :1] + pairs[..., 1:]).flatten(-2)


def plain_write(cache, k, v, at, case):
    kc, vc, pairs = (c.movedim(1, 3) for c in cells(cache, case))  # [pages, tiles, 16, heads, bytes]
    (kq, kp), (vq, vp) = quantise(k, case), quantise(v, case)
    kc[at], vc[at], pairs[at] = kq, vq, torch.cat((kp, vp), -1)


def plain_read(cache, at, case):
    kc, vc, pairs = (c.movedim(1, 3)[at] for c in cells(cache, case))
    half = pairs.shape[-1] // 2
    return values(kc, pairs[..., :half], case).bfloat16(), values(vc, pairs[..., half:], case).bfloat16()


def plain_attention(q, cache, table, lens, case):
    B, n, _, D = q.shape
    H = cache.shape[1]
    got = cells(cache[table.long()].flatten(0, 1), case)
    # [B * width, heads, tiles, 16, ..] -> [B, heads, positions, ..]
    kc, vc, pairs = (c.unflatten(0, (B, -1)).transpose(1, 2).flatten(2, 4) for c in got)
    half = pairs.shape[-1] // 2
    pos = torch.arange(kc.shape[2], device=q.device)
    end = lens.long()[:, None] - n + 1 + torch.arange(n, device=q.device)  # [B, n]: the first position that is not seen
    seen = pos < end[..., None]
    if case["window"]:
        seen &= pos >= end[..., None] - case["window"]
    k = values(kc, pairs[..., :half], case)
    rows = q.float().unflatten(2, (H, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, heads, n * group, D]
    s = rows @ k.transpose(-1, -2) / math.sqrt(D)
    del k
    s = s.unflatten(2, (n, -1)).masked_fill(~seen[:, None, :, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = (s - top.masked_fill(top == float("-inf"), 0)).exp().flatten(2, 3)
    del s
    v = values(vc, pairs[..., half:], case).masked_fill(~seen.any(1)[:, None, :, None], 0)
    total = p.sum(-1, keepdim=True)
    out = p @ v / torch.where(total == 0, torch.ones_like(total), total)
    return out.unflatten(2, (n, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3).bfloat16()


# The definition in 64 bits, a sequence at a time


def exact(case, seed):
    state = prepare(case, seed)
    H, D, G, bits, page = case["heads"], case["D"], case["G"], case["bits"], case["page"]
    rb, tb = D * bits // 8, token_bytes(case)
    raw = state["cache"]
    table, lens = state["table"].tolist(), state["lens"].tolist()

    def unpack(byte):
        if bits == 8:
            return byte.double()
        return torch.stack([(byte >> sh & 15).double() for sh in (0, 4)], -1).reshape(*byte.shape[:-1], -1)

    def cached(b, first, last):
        """K and V [tokens, heads, D] of positions first .. last - 1 of sequence b."""
        ids = torch.tensor(table[b][first // page : -(-last // page)], device="cuda")
        t = raw[ids].view(len(ids), H, page // 16, 16 * tb)
        found = []
        for which in (0, 1):
            codes = unpack(t[..., which * 16 * rb : (which + 1) * 16 * rb]).view(len(ids), H, page, D)
            meta = t[..., 32 * rb :].contiguous().view(torch.float16).double().view(len(ids), H, page, 2, D // G, 2)[:, :, :, which]
            x = codes.view(len(ids), H, page, D // G, G) * meta[..., 0, None] + meta[..., 1, None]
            skip = first - first // page * page
            found.append(x.view(len(ids), H, page, D).transpose(1, 2).reshape(-1, H, D)[skip : skip + last - first])
        return found

    if case["op"] == "attend":
        n, rep = case["tokens"], case["q_heads"] // H
        out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
        for b, length in enumerate(lens):
            for j in range(n):
                at = length - n + j
                if at < 0:
                    continue
                first = max(0, at - case["window"] + 1) if case["window"] else 0
                k, v = cached(b, first, at + 1)
                q = state["q"][b, j].double().view(H, rep, D)
                w = torch.softmax(torch.einsum("hrd,thd->hrt", q, k) * D**-0.5, -1)
                out[b, j] = torch.einsum("hrt,thd->hrd", w, v).reshape(-1, D)
        return out
    if case["op"] == "read":
        parts = [cached(b, 0, length) for b, length in enumerate(lens)]
        return tuple(torch.cat([p[i] for p in parts]) for i in (0, 1))

    def stored(x):
        """x's groups through their stored scales, biases and codes; every step of the definition that rounds is rounded here."""
        x = x.double().unflatten(-1, (-1, G))
        low, high = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
        top = 2.0**bits - 1
        scale = ((high - low).float().double() / top).float().half().double()
        bias = low.half().double()
        ratio = ((x - bias).float().double() / scale).float().double()
        code = torch.where(scale > 0, torch.clamp(torch.round(ratio), 0.0, top), torch.zeros_like(ratio))
        return (code * scale + bias).flatten(-2)

    return stored(state["k"]), stored(state["v"])
