"""Workloads of the paged cache in 8 bits, of positions with several axes and of shaped scores, in a plain form and
through the library.

A target model's cache may hold its keys and values in e4m3 with a scale for each head: ``append`` quantises them as it
rotates and writes them, ``attend`` reads them under the tree's attention, ``read`` gives them back in 16 bits.  Models of
images and video rotate by positions of several axes (``append`` with ``axes``), others cap their scores with a tanh, look
back over a window, or add a bias that grows with the distance (``attend`` with ``cap``, ``window``, ``alibi``).  ``run``
computes one pass in elementary torch operations in 32 bits, rounded once, or, when ``own`` is true, through this
repository's package; ``exact`` states the same results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
SECTIONS = {128: (16, 24, 24), 64: (8, 12, 12)}  # pairs of a head that turn by time, height and width


# ------------------------------------------------------------------------------------------------------------- cases
def _case(name, op, batch, slots, ctx, q_heads, kv_heads, dim, page, **more):
    return {"name": name, "op": op, "batch": batch, "slots": slots, "ctx": ctx, "prefix": 0, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "type": "bf16", "layout": "head", "cache": "e4m3",
            "axes": False, "cap": 0.0, "window": 0, "alibi": False, **more}


def listed():
    return [
        # one token of one request after a short prompt: the latency of a call
        _case("append8_b1_s1", "append", 1, 1, 117, 32, 8, 128, 16),
        # a static tree of 61 slots for each of 16 requests behind images: positions of three axes, an 8-bit cache
        _case("append8_axes_b16_s61", "append", 16, 61, 2048, 32, 8, 128, 64, axes=True),
        # the prompts of four requests with images, 16-bit cache, token-major pages, half precision
        _case("append_axes_b4_s4096", "append", 4, 4096, 0, 40, 8, 128, 16, axes=True, cache="same", layout="token", type="f16"),
        # the prefill of a 32K-token history into an 8-bit cache
        _case("append8_b1_s32768", "append", 1, 32768, 0, 32, 8, 128, 128),
        # the newest tokens of 64 requests, handed to a model that keeps its own 16-bit cache
        _case("read8_b64_t61", "read", 64, 61, 1000, 40, 8, 128, 16),
        # a 32K-token history read back whole
        _case("read8_b1_t32768", "read", 1, 32768, 0, 32, 8, 128, 64),
        # one token of one request after a short prompt
        _case("attend8_b1_s1_c117", "attend", 1, 1, 117, 32, 8, 128, 16),
        # plain decoding, 64 requests behind one long system prompt: bound by the cache's bytes
        _case("attend8_b64_s1_p8192", "attend", 64, 1, 1024, 32, 8, 128, 64, prefix=8192),
        # static trees of 61 slots, 16 requests behind a prompt that ends inside a page
        _case("attend8_b16_s61_p12001", "attend", 16, 61, 2048, 32, 8, 128, 64, prefix=12001),
        # one token of a model that caps its scores and looks back 1024 tokens, half precision, heads of 64
        _case("attend_cap_window_b1_s1_c1500", "attend", 1, 1, 1500, 16, 8, 64, 16, cache="same", cap=50.0, window=1024,
              type="f16"),
        # its trees of 61 slots for 16 requests, a window of 4096
        _case("attend_cap_window_b16_s61_c8192", "attend", 16, 61, 8192, 32, 8, 128, 64, cache="same", cap=50.0, window=4096),
        # block drafts of 17 slots of a model without rotations, whose scores fall with the distance; a key head a query head
        _case("attend_alibi_b8_s17_c4096", "attend", 8, 17, 4096, 32, 32, 128, 16, cache="same", alibi=True),
    ]


def _log_int(rng, low, high):
    return min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("append", "read", "attend", "attend", "attend"))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8))
    more = {"type": rng.choice(("bf16", "bf16", "f16")), "layout": rng.choice(("head", "token")),
            "cache": rng.choice(("e4m3", "e4m3", "same"))}
    heads = (group * kv_heads, kv_heads, rng.choice((64, 128, 128)), rng.choice((8, 16, 32, 64, 128)))
    if op in ("append", "read"):
        batch = _log_int(rng, 1, 64)
        slots = _log_int(rng, 1, 32768 // batch)
        more["axes"] = op == "append" and (more["cache"] == "same" or rng.random() < 0.4)
        return _case("drawn", op, batch, slots, _log_int(rng, 1, 4096), *heads, **more)
    slots = rng.choice((1, 1, 17, 61, rng.randint(2, 64)))
    batch = _log_int(rng, 1, 64 if slots <= 17 else 16)
    # at most as many rows times keys as the largest listed case has
    most = 4.0e8 / (batch * slots * group * kv_heads)
    more["prefix"] = rng.choice((0, 1)) * _log_int(rng, 1, max(1, min(32768, int(most * 0.6))))
    ctx = _log_int(rng, 1, max(1, min(32768, int(most * 0.3), 400000 // batch)))
    kind = rng.choice(("cap", "window", "alibi", "cap window")) if more["cache"] == "same" or rng.random() < 0.4 else ""
    more["cap"] = rng.choice((20.0, 30.0, 50.0)) if "cap" in kind else 0.0
    more["window"] = _log_int(rng, 2, 8192) if "window" in kind else 0
    more["alibi"] = kind == "alibi"
    return _case("drawn", op, batch, slots, ctx, *heads, **more)


# ------------------------------------------------------------------------------------------------------------ inputs
def _lengths(batch, most, least):
    """Lengths of the requests: the first has `most`, the others lie between half of it and it."""
    return [max(least, most - int((most // 2) * ((b * 0.618034) % 1.0))) for b in range(batch)]


def _valid(batch, slots):
    """Slots of each tree that hold a node: a few requests end in up to 4 pad slots."""
    return [max(1, slots - (b * 7 % 5 if 8 <= slots <= 64 and b % 3 == 2 else 0)) for b in range(batch)]


def _trees(rng, batch, slots):
    """Random trees (parents before children, pads at the end): depth (-1 = pad) and ancestor mask of a slot."""
    depth = np.full((batch, slots), -1, np.int32)
    mask = np.zeros((batch, slots), np.uint64)
    rows = np.arange(batch)
    valid = np.array(_valid(batch, slots))
    depth[:, 0], mask[:, 0] = 0, 1
    for i in range(1, slots):
        p = np.maximum(0, i - 1 - np.floor(rng.exponential(4.0, batch)).astype(np.int64))
        on = i < valid
        depth[:, i] = np.where(on, depth[rows, p] + 1, -1)
        mask[:, i] = np.where(on, mask[rows, p] | np.uint64(1 << i), np.uint64(0))
    return depth, mask


def _gpu(x, dtype=None):
    x = torch.from_numpy(np.ascontiguousarray(x))
    return (x if dtype is None else x.to(dtype)).to(DEV)


def _pages_of(tokens, page):
    return -(-tokens // page)


def _cache_plan(case, rng):
    """Page tables: the shared prefix's pages and each request's, in no order, and the number of pages."""
    batch, page = case["batch"], case["page"]
    own_pages = _pages_of(case["ctx"] + case["slots"], page)
    prefix_pages = _pages_of(case["prefix"], page)
    total = batch * own_pages + prefix_pages + 3
    order = rng.permutation(total)[:total - 3].astype(np.int32)
    return order[:prefix_pages], order[prefix_pages:].reshape(batch, own_pages), total


def _cache_shape(case, pages):
    if case["layout"] == "token":
        return pages, case["page"], case["kv_heads"], case["dim"]
    return pages, case["kv_heads"], case["page"], case["dim"]


def _caches(case, pages, gen):
    """Keys and values of unit variance, and each head's scale: its largest magnitudes come near e4m3's."""
    shape, heads = _cache_shape(case, pages), case["kv_heads"]
    s = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=TYPES[case["type"]])
        if case["cache"] == "e4m3":
            scale = 0.012 + 0.008 * torch.rand(heads, generator=gen, device=DEV)
            by_head = scale.view((heads, 1) if case["layout"] == "token" else (heads, 1, 1))
            x = torch.cat([(part.float() / by_head).clamp(-448, 448).to(E4M3).view(torch.uint8) for part in x.split(256)]).view(E4M3)
            s[name + "_scale"] = scale
        s[name + "_cache"] = x
    return s


def _handle(case, pages):
    import hybrid_draft_tree_gb300 as g
    kv = g.GraftKV(g.graft_kv_default_config(
        case["q_heads"], case["kv_heads"], case["dim"], case["page"], pages, case["batch"], min(64, case["slots"]),
        g.GRAFT_F16 if case["type"] == "f16" else g.GRAFT_BF16, layout=case["layout"],
        cache=None if case["cache"] == "same" else case["cache"]))
    if case["axes"]:
        kv.set_axes(np.repeat(np.arange(3), SECTIONS[case["dim"]]).tolist())
    return kv


def _image_positions(slots):
    """Positions [3, slots] of a prompt of text with images of 24 by 32 patches in it: text moves all axes on together, a
    patch lies at its image's time, row and column."""
    pos = np.zeros((3, slots), np.int64)
    at, now, patches = 0, 0, 24 * 32
    while at < slots:
        n = min(100, slots - at)
        pos[:, at:at + n] = now + np.arange(n)
        at, now = at + n, now + n
        n = min(patches, slots - at)
        i = np.arange(n)
        pos[:, at:at + n] = now + np.stack([0 * i, i // 32, i % 32])
        at, now = at + n, now + 32
    return pos


def _prepare_append(case, rng, gen):
    batch, slots, dim, dtype = case["batch"], case["slots"], case["dim"], TYPES[case["type"]]
    widths = [case["q_heads"] * dim, case["kv_heads"] * dim, case["kv_heads"] * dim]
    _, table, pages = _cache_plan(case, rng)
    # the projections come as column ranges of one matrix
    q, k, v = torch.randn((batch * slots, sum(widths)), generator=gen, device=DEV, dtype=dtype).split(widths, 1)
    ctx = np.array(_lengths(batch, case["ctx"], 0), np.int32)
    s = {"q": q, "k": k, "v": v, "table": _gpu(table), "ctx_len": _gpu(ctx), "depth": None, "positions": None,
         **_caches(case, pages, gen)}
    depth = np.tile(np.arange(slots, dtype=np.int32), (batch, 1))
    if slots <= 64:
        depth, _ = _trees(rng, batch, slots)
        s["depth"] = _gpu(depth)
    length = case["ctx"] + slots
    if case["axes"]:
        if slots <= 64:  # text behind images, whose positions run behind the cache's places
            pos = np.broadcast_to(np.maximum(depth, 0) + (ctx - ctx // 3)[:, None], (3, batch, slots))
        else:
            pos = _image_positions(slots)[:, None] + ctx[:, None]
        s["positions"] = _gpu(pos.astype(np.int32))
    angle = np.arange(length)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    s["rope"] = _gpu(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    s["q_out"] = torch.zeros((batch * slots, widths[0]), device=DEV, dtype=dtype)
    if own:
        s["kv"] = _handle(case, pages)
    return s


def _prepare_read(case, rng, gen):
    batch, slots = case["batch"], case["slots"]
    _, table, pages = _cache_plan(case, rng)
    first = _lengths(batch, case["ctx"], 0)
    s = {"table": _gpu(table), "first": _gpu(np.array(first, np.int32)),
         "count": _gpu(np.array(_lengths(batch, slots, 1), np.int32)), **_caches(case, pages, gen)}
    for name in ("k_out", "v_out"):
        s[name] = torch.zeros((batch * slots, case["kv_heads"] * case["dim"]), device=DEV, dtype=TYPES[case["type"]])
    if own:
        s["kv"] = _handle(case, pages)
    return s


def _prepare_attend(case, rng, gen):
    batch, slots, dim, dtype = case["batch"], case["slots"], case["dim"], TYPES[case["type"]]
    prefix_pages, table, pages = _cache_plan(case, rng)
    _, mask = _trees(rng, batch, slots)
    # queries of unit variance give scores of variance 1, flatter than trained heads: 2.5 times that; before a cap, which
    # is there because scores grow large, 10 times
    q = torch.randn((batch * slots, case["q_heads"] * dim), generator=gen, device=DEV, dtype=dtype) * (10 if case["cap"] else 2.5)
    s = {"q": q, **_caches(case, pages, gen), "table": _gpu(table),
         "prefix_pages": _gpu(prefix_pages) if case["prefix"] else None,
         "ctx_len": _gpu(np.array(_lengths(batch, case["ctx"], 0), np.int32)), "mask": _gpu(mask.view(np.int64)),
         "out": torch.zeros_like(q), "lse": torch.zeros((batch * slots, case["q_heads"]), device=DEV), "slopes": None}
    if case["alibi"]:  # a geometric series over the heads, from 2^(-8 / heads) to 2^-8
        s["slopes"] = _gpu(2.0 ** (-8.0 * np.arange(1, case["q_heads"] + 1) / case["q_heads"]), torch.float32)
    if own:
        s["kv"] = _handle(case, pages)
    return s


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    make = {"append": _prepare_append, "read": _prepare_read, "attend": _prepare_attend}[case["op"]]
    return {**make(case, rng, gen), "case": case}


# --------------------------------------------------------------------------------------------------------- one pass
def _by_token(cache, case):
    """A view [pages, page, kv_heads, dim] of a cache of either layout; 8-bit elements as bytes, which can be indexed."""
    cache = cache.view(torch.uint8) if cache.dtype == E4M3 else cache
    return cache if case["layout"] == "token" else cache.transpose(1, 2)


def _values(x, s, name):
    """What elements [..., kv_heads, dim] of a cache stand for, in 32 bits."""
    return x.view(E4M3).float() * s[name + "_scale"][:, None] if x.dtype == torch.uint8 else x.float()


def _plain_append(s):
    case = s["case"]
    batch, slots, dim, page, half = case["batch"], case["slots"], case["dim"], case["page"], case["dim"] // 2
    index = torch.arange(slots, device=DEV).expand(batch, slots)
    depth = index if s["depth"] is None else s["depth"].long()
    base = s["ctx_len"].long()[:, None]
    if case["axes"]:
        axis = torch.repeat_interleave(torch.arange(3, device=DEV), torch.tensor(SECTIONS[dim], device=DEV), output_size=half)
        place = s["positions"].long().view(3, -1).t()[:, axis]                          # [tokens, pairs]
        pair = torch.arange(half, device=DEV)
        cos, sin = s["rope"][place, pair][:, None], s["rope"][place, pair + half][:, None]
    else:
        cs = s["rope"][(base + depth.clamp(min=0)).view(-1)][:, None]
        cos, sin = cs[..., :half], cs[..., half:]

    def turn(x):
        x = x.float().reshape(batch * slots, -1, dim)
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    live = (depth >= 0).view(-1, 1)
    at = base + index
    pages, offset = s["table"].long().gather(1, at // page).view(-1), (at % page).view(-1)
    for name, x in (("k", turn(s["k"])), ("v", s["v"].float().reshape(batch * slots, -1, dim))):
        cache = _by_token(s[name + "_cache"], case)
        if case["cache"] == "e4m3":
            x = (x / s[name + "_scale"][:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        # a pad's place keeps what it held
        cache[pages, offset] = torch.where(live[..., None], x.to(cache.dtype), cache[pages, offset])
    s["q_out"].copy_(torch.where(live, turn(s["q"]).flatten(1), 0.0))
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_read(s):
    case = s["case"]
    batch, slots, page = case["batch"], case["slots"], case["page"]
    index = torch.arange(slots, device=DEV)
    live = index < s["count"][:, None]
    at = s["first"].long()[:, None] + torch.where(live, index, 0)
    pages, offset = s["table"].long().gather(1, at // page), at % page
    for name in ("k", "v"):
        x = _values(_by_token(s[name + "_cache"], case)[pages, offset], s, name)
        s[name + "_out"].copy_(torch.where(live[..., None, None], x, 0.0).view(batch * slots, -1))
    return s["k_out"], s["v_out"]


def _plain_attend(s):
    case = s["case"]
    batch, slots, prefix, page = case["batch"], case["slots"], case["prefix"], case["page"]
    hk, dim, group = case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    keys, rows = case["ctx"] + slots, slots * group
    # [kv head, request, slot and query head of the group, dim]
    q = s["q"].float().view(batch, slots, hk, group, dim).permute(2, 0, 1, 3, 4).reshape(hk, batch, rows, dim)
    slot = torch.arange(slots, device=DEV)
    bits = (s["mask"][:, :, None] >> slot) & 1                                           # [batch, slots, slots]
    count = bits.sum(-1)
    live = count > 0
    # a slot follows the context as if its path had been emitted token by token
    here = prefix + s["ctx_len"].long()[:, None]
    place = here + count - 1                                                             # [batch, slots]
    slopes = None if s["slopes"] is None else s["slopes"].view(hk, 1, 1, group, 1)

    def shaped(score, distance, seen):
        """Scores [hk, batch, rows, keys] capped, biased and masked; distance, seen: [batch, slots, keys]."""
        if case["cap"]:
            score = case["cap"] * torch.tanh(score / case["cap"])
        if slopes is not None:
            score = (score.view(hk, batch, slots, group, -1) - slopes * distance[:, :, None].float()).view(score.shape)
        if case["window"]:
            seen = seen & (distance < case["window"])
        return score.masked_fill(~seen.repeat_interleave(group, 1), -math.inf)

    at = torch.arange(keys, device=DEV)
    pages = s["table"].long()[:, at // page]
    k, v = (_values(_by_token(s[name + "_cache"], case)[pages, at % page], s, name).permute(2, 0, 1, 3) for name in ("k", "v"))
    node = at - s["ctx_len"].long()[:, None]                                             # [batch, keys]: slot of a key
    of_node = node.clamp(0, slots - 1)[:, None, :].expand(batch, slots, keys)
    seen = (node < 0)[:, None, :] | ((node < slots)[:, None, :] & (bits.gather(2, of_node) == 1))
    rank = (bits.cumsum(-1) - bits).gather(2, of_node)                                   # seen slots before a key's
    key_place = torch.where((node < 0)[:, None, :], prefix + at, here[:, :, None] + rank)
    score = shaped((q @ k.transpose(-1, -2)) / math.sqrt(dim), place[:, :, None] - key_place, seen & live[:, :, None])
    if prefix:
        at = torch.arange(prefix, device=DEV)
        pages = s["prefix_pages"].long()[at // page]
        pk, pv = (_values(_by_token(s[name + "_cache"], case)[pages, at % page], s, name).transpose(0, 1) for name in ("k", "v"))
        first = (q.flatten(1, 2) @ pk.transpose(-1, -2)).view(hk, batch, rows, prefix) / math.sqrt(dim)
        score = torch.cat([shaped(first, place[:, :, None] - at, live[:, :, None].expand(-1, -1, prefix)), score], -1)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = (score - top).exp()
    total = e.sum(-1, keepdim=True)
    out = e[..., prefix:] @ v
    if prefix:
        out = out + (e[..., :prefix].flatten(1, 2) @ pv).view(out.shape)
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    s["out"].copy_(out.view(hk, batch, slots, group, dim).permute(1, 2, 0, 3, 4).reshape(batch * slots, -1))
    s["lse"].copy_(lse.view(hk, batch, slots, group).permute(1, 2, 0, 3).reshape(batch * slots, -1))
    return s["out"], s["lse"]


def run(s):
    case = s["case"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[case["op"]](s)
    batch, slots = case["batch"], case["slots"]
    scales = {name: s[name] for name in ("k_scale", "v_scale")} if case["cache"] == "e4m3" else {}
    if case["op"] == "append":
        s["kv"].append(batch, slots, s["q"], s["k"], s["v"], s["rope"], s["table"], s["ctx_len"], s["k_cache"], s["v_cache"],
                       s["q_out"], pos=s["depth"], positions=s["positions"], **scales)
        return s["q_out"], s["k_cache"], s["v_cache"]
    if case["op"] == "read":
        s["kv"].read(batch, slots, s["k_cache"], s["v_cache"], s["table"], s["first"], s["count"], s["k_out"], s["v_out"], **scales)
        return s["k_out"], s["v_out"]
    s["kv"].attend(batch, slots, s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx_len"], case["ctx"], s["out"],
                   prefix_pages=s["prefix_pages"], prefix_len=case["prefix"], tree_mask=s["mask"], lse=s["lse"],
                   softcap=case["cap"], window=case["window"], slopes=s["slopes"], **scales)
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------------------------- what a pass costs
def work(case):
    batch, slots = case["batch"], case["slots"]
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    size = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        tokens = sum(_valid(batch, slots))
        # angles, depth and positions of a token beside its rows
        return {"bytes": tokens * (dim * (hq * 4 + 2 * hk * (2 + size) + 4) + 4 + 12 * case["axes"]),
                "flops": tokens * (hq + hk) * dim * 3 + tokens * 2 * hk * dim * (size == 1)}
    if case["op"] == "read":
        tokens = sum(_lengths(batch, slots, 1))
        return {"bytes": tokens * 2 * hk * dim * (size + 2), "flops": tokens * 2 * hk * dim * (size == 1)}
    ctx, valid = _lengths(batch, case["ctx"], 0), _valid(batch, slots)
    window, prefix = case["window"] or 1 << 40, case["prefix"]
    # keys that some slot sees: the prefix's once, of a request the last `window` and its slots; a tree's path has about 4
    far = min(prefix, max(0, window - min(ctx)))
    keys = far + sum(min(c, window) for c in ctx) + sum(valid)
    pairs = sum(n * min(prefix + c + min(slots, 4), window) for n, c in zip(valid, ctx))
    return {"bytes": keys * hk * dim * size * 2 + batch * slots * (hq * (dim * 4 + 4) + 8), "flops": 4 * pairs * hq * dim}


# ------------------------------------------------------------------------------------------- the definition in 64 bits
def _nearest(x):
    """The e4m3 numbers next to x (ties to an even last bit): three bits after the leading one, steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    case = s["case"]
    batch, slots, dim, page = case["batch"], case["slots"], case["dim"], case["page"]
    ctx, table, rope = s["ctx_len"].cpu().numpy().astype(np.int64), s["table"].cpu().numpy(), s["rope"].double()
    depth = np.tile(np.arange(slots), (batch, 1)) if s["depth"] is None else s["depth"].cpu().numpy().astype(np.int64)
    b, i = np.nonzero(depth >= 0)
    rows = _gpu(b * slots + i)
    place = np.repeat((ctx[b] + depth[b, i])[:, None], dim // 2, 1)
    if case["axes"]:
        pos = s["positions"].cpu().numpy().astype(np.int64)
        place = np.concatenate([np.repeat(pos[a][b, i][:, None], n, 1) for a, n in enumerate(SECTIONS[dim])], 1)
    place, pair = _gpu(place), torch.arange(dim // 2, device=DEV)
    turn = torch.complex(rope[place, pair], rope[place, pair + dim // 2])[:, None]

    def turned(x):
        x = x[rows].double().view(len(b), -1, dim)
        z = torch.complex(x[..., :dim // 2].contiguous(), x[..., dim // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    at = ctx[b] + i
    pages, offset = _gpu(table[b, at // page].astype(np.int64)), _gpu(at % page)
    caches = []
    for name, new in (("k", turned(s["k"])), ("v", s["v"][rows].double().view(len(b), -1, dim))):
        cache = s[name + "_cache"].double()
        if case["cache"] == "e4m3":
            new = _nearest(new / s[name + "_scale"].double()[:, None])
        _by_token(cache, case)[pages, offset] = new
        caches.append(cache)
    q = torch.zeros((batch * slots, case["q_heads"] * dim), device=DEV, dtype=torch.float64)
    q[rows] = turned(s["q"]).flatten(1)
    return (q, *caches)


def _exact_read(s):
    case = s["case"]
    batch, slots, page, width = case["batch"], case["slots"], case["page"], case["kv_heads"] * case["dim"]
    table, first, count = (s[name].cpu().numpy().astype(np.int64) for name in ("table", "first", "count"))
    found = []
    for name in ("k", "v"):
        out = torch.zeros((batch, slots, width), device=DEV, dtype=torch.float64)
        cache = _by_token(s[name + "_cache"], case)
        for b in range(batch):
            at = first[b] + np.arange(count[b])
            x = cache[_gpu(table[b, at // page]), _gpu(at % page)]
            x = x.view(E4M3).double() * s[name + "_scale"].double()[:, None] if case["cache"] == "e4m3" else x.double()
            out[b, :count[b]] = x.flatten(1)
        found.append(out.view(batch * slots, width))
    return tuple(found)


def _exact_attend(s):
    case = s["case"]
    batch, slots, prefix, page = case["batch"], case["slots"], case["prefix"], case["page"]
    hk, dim, group = case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros((batch, slots, hk, group, dim), device=DEV, dtype=torch.float64)
    lse = torch.full((batch, slots, hk, group), -math.inf, device=DEV, dtype=torch.float64)
    table, ctx = s["table"].cpu().numpy(), s["ctx_len"].cpu().numpy()
    mask = s["mask"].cpu().numpy().view(np.uint64)
    shared = np.empty(0, np.int64)
    if prefix:
        shared = s["prefix_pages"].cpu().numpy().astype(np.int64).repeat(page)[:prefix] * page + np.arange(prefix) % page
    caches = [_by_token(s[name + "_cache"], case).flatten(0, 1) for name in ("k", "v")]
    q = s["q"].view(batch, slots, hk, group, dim)
    for b in range(batch):
        c = int(ctx[b])
        places = np.concatenate([shared, table[b].astype(np.int64).repeat(page)[:c + slots] * page + np.arange(c + slots) % page])
        k, v = (x[_gpu(places)] for x in caches)
        if case["cache"] == "e4m3":
            k, v = (x.view(E4M3).double() * s[n].double()[:, None] for x, n in ((k, "k_scale"), (v, "v_scale")))
        k, v = k.double(), v.double()
        # positions, slot by slot: the keys before the tree in order, then the slots of the path in order
        seen = np.zeros((slots, prefix + c + slots), bool)
        distance = np.zeros((slots, prefix + c + slots), np.int64)
        for i in range(slots):
            path = [j for j in range(slots) if int(mask[b, i]) >> j & 1]
            if path:
                at = np.concatenate([np.arange(prefix + c), prefix + c + np.array(path)])
                distance[i, at] = len(at) - 1 - np.arange(len(at))
                seen[i, at] = distance[i, at] < (case["window"] or 1 << 40)
        score = torch.einsum("shgd,nhd->hgsn", q[b].double(), k) * dim ** -0.5
        if case["cap"]:
            score = torch.tanh(score / case["cap"]) * case["cap"]
        if s["slopes"] is not None:
            score -= s["slopes"].double().view(hk, group, 1, 1) * _gpu(distance).double()
        score.masked_fill_(~_gpu(seen), -math.inf)
        on = _gpu(np.nonzero(mask[b])[0])
        z = torch.logsumexp(score[:, :, on], -1)
        weight = torch.exp(score[:, :, on] - z[..., None])
        out[b, on] = torch.einsum("hgsn,nhd->shgd", weight, v)
        lse[b, on] = z.permute(2, 0, 1)
    return out.view(batch * slots, -1), lse.view(batch * slots, -1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)
