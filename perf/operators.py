"""Workloads of the operators around the draft tree's verification, each in a plain form and through the library.

Three operators make the target's side of a decode step: keys and values of the tree's slots appended to a paged cache
with the position rotation applied on the way (``append``), attention of the tree's slots over that cache, where the
requests share a long prefix (``attend``), and penalties, biases and grammar masks on the tree's logits before they are
verified (``logits``).  ``run`` computes one pass in elementary torch operations in 32 bits, rounded once, or, when
``own`` is true, through this repository's package; ``exact`` states the same results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------------------- cases
def _append(name, batch, slots, ctx, q_heads, kv_heads, dim, page, **more):
    return {"name": name, "op": "append", "batch": batch, "slots": slots, "ctx": ctx, "prefix": 0, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "type": "bf16", "layout": "head", "rot": dim,
            "interleaved": False, "accepted": False, "qkv": True, **more}


def _attend(name, batch, slots, prefix, ctx, q_heads, kv_heads, dim, page, **more):
    return {"name": name, "op": "attend", "batch": batch, "slots": slots, "prefix": prefix, "ctx": ctx,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "type": "bf16", "layout": "head", **more}


def _logits(name, batch, slots, vocab, hist, type_, **more):
    return {"name": name, "op": "logits", "batch": batch, "slots": slots, "vocab": vocab, "hist": hist, "type": type_,
            "bias": 64, "grammar": 8, "pad": 0, **more}


def listed():
    return [
        # one token of one request after a short prompt: the latency of a call
        _append("append_b1_s1", 1, 1, 117, 32, 8, 128, 16),
        # a static tree of 61 slots for each of 16 requests, projected as one fused q|k|v row per slot
        _append("append_b16_s61", 16, 61, 2048, 32, 8, 128, 64),
        # the accepted paths of 64 block drafts of 16 tokens written again at contiguous positions, no queries
        _append("append_b64_s17_accepted", 64, 17, 1000, 40, 8, 128, 16, accepted=True, layout="token", type="f16"),
        # the prefill of a 32K-token history, half of each head rotated, neighbouring elements paired
        _append("append_b1_s32768", 1, 32768, 0, 32, 8, 128, 128, rot=64, interleaved=True),
        # one token of one request after a short prompt
        _attend("attend_b1_s1_c117", 1, 1, 0, 117, 32, 8, 128, 16),
        # plain decoding, 64 requests behind one long system prompt: bound by the cache's bytes
        _attend("attend_b64_s1_p8192", 64, 1, 8192, 1024, 32, 8, 128, 64),
        # static trees of 61 slots, 16 requests behind a prompt that ends inside a page
        _attend("attend_b16_s61_p12001", 16, 61, 12001, 2048, 32, 8, 128, 64),
        # block drafts of 17 slots, 64 requests, heads of 64 in half precision, token-major pages
        _attend("attend_b64_s17_p2048_f16", 64, 17, 2048, 777, 40, 8, 64, 16, type="f16", layout="token"),
        # one tree of 61 slots at the end of a 32K-token history
        _attend("attend_b1_s61_c32768", 1, 61, 0, 32768, 32, 8, 128, 16),
        # one token's fp32 row of a small vocabulary: the latency of a call
        _logits("logits_b1_s1_v32000", 1, 1, 32000, 300, "f32"),
        # static trees of 16 requests, every rule on
        _logits("logits_b16_s61_v151936", 16, 61, 151936, 4096, "bf16"),
        # block drafts of 64 requests with long histories, rows that start off 16-byte boundaries
        _logits("logits_b64_s17_v128256_odd", 64, 17, 128256, 8192, "bf16", pad=3),
    ]


def _log_int(rng, low, high):
    return min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "logits"))
    type_ = rng.choice(("bf16", "bf16", "f16"))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8))
    dim = rng.choice((64, 128, 128))
    page = rng.choice((8, 16, 32, 64, 128))
    layout = rng.choice(("head", "token"))
    if op == "append":
        batch = _log_int(rng, 1, 64)
        slots = _log_int(rng, 1, 32768 // batch)
        rot = rng.choice((dim, dim, dim // 2))
        return _append(None, batch, slots, _log_int(rng, 1, 4096), group * kv_heads, kv_heads, dim, page, type=type_,
                       layout=layout, rot=rot, interleaved=rng.random() < 0.3,
                       accepted=2 <= slots <= 64 and rng.random() < 0.4, qkv=rng.random() < 0.7) | {"name": "drawn"}
    if op == "attend":
        slots = rng.choice((1, 1, 17, 61, rng.randint(2, 64)))
        batch = _log_int(rng, 1, 64 if slots <= 17 else 16)
        # at most as many rows times keys as the largest listed case has
        most = 4.0e8 / (batch * slots * group * kv_heads)
        prefix = rng.choice((0, 1)) * _log_int(rng, 1, max(1, min(32768, int(most * 0.6))))
        ctx = _log_int(rng, 1, max(1, min(32768, int(most * 0.3), 400000 // batch)))
        return _attend(None, batch, slots, prefix, ctx, group * kv_heads, kv_heads, dim, page, type=type_,
                       layout=layout) | {"name": "drawn"}
    slots = rng.choice((1, 17, 61, rng.randint(2, 64)))
    vocab = rng.choice((32000, 128256, 151936, _log_int(rng, 1000, 151936)))
    batch = _log_int(rng, 1, max(1, min(64, 140_000_000 // (slots * vocab * 2))))
    return _logits(None, batch, slots, vocab, _log_int(rng, 1, 32768 if batch <= 16 else 8192),
                   rng.choice(("bf16", "bf16", "f32")), bias=rng.choice((0, 5, 300)), grammar=rng.choice((0, 1, 8)),
                   pad=rng.choice((0, 0, 1, 8))) | {"name": "drawn"}


# ------------------------------------------------------------------------------------------------------------ inputs
def _lengths(batch, most, least):
    """Lengths of the requests: the first has `most`, the others lie between half of it and it."""
    return [max(least, most - int((most // 2) * ((b * 0.618034) % 1.0))) for b in range(batch)]


def _valid(batch, slots):
    """Slots of each tree that hold a node: a few requests end in up to 4 pad slots."""
    return [max(1, slots - (b * 7 % 5 if slots >= 8 and b % 3 == 2 else 0)) for b in range(batch)]


def _trees(rng, batch, slots):
    """Random trees (parents before children, pads at the end): parent, depth (-1 = pad) and ancestor mask of a slot."""
    parent = np.full((batch, slots), -1, np.int64)
    depth = np.full((batch, slots), -1, np.int32)
    mask = np.zeros((batch, slots), np.uint64)
    rows = np.arange(batch)
    valid = np.array(_valid(batch, slots))
    depth[:, 0], mask[:, 0] = 0, 1
    for i in range(1, slots):
        p = np.maximum(0, i - 1 - np.floor(rng.exponential(4.0, batch)).astype(np.int64))
        on = i < valid
        parent[:, i] = np.where(on, p, -1)
        depth[:, i] = np.where(on, depth[rows, p] + 1, -1)
        mask[:, i] = np.where(on, mask[rows, p] | np.uint64(1 << i), np.uint64(0))
    return parent, depth, mask


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


def _cache(case, pages, gen, dtype):
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["layout"] == "token":
        shape = (pages, case["page"], case["kv_heads"], case["dim"])
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _kv_handle(case, pages):
    import hybrid_draft_tree_gb300 as g
    over = {"rot_dim": case["rot"], "rot_interleaved": int(case["interleaved"])} if case["op"] == "append" else {}
    return g.GraftKV(g.graft_kv_default_config(
        case["q_heads"], case["kv_heads"], case["dim"], case["page"], pages, case["batch"], min(64, case["slots"]),
        g.GRAFT_F16 if case["type"] == "f16" else g.GRAFT_BF16, layout=case["layout"], **over))


def _prepare_append(case, rng, gen):
    batch, slots, dim, dtype = case["batch"], case["slots"], case["dim"], TYPES[case["type"]]
    widths = [case["q_heads"] * dim, case["kv_heads"] * dim, case["kv_heads"] * dim]
    _, table, pages = _cache_plan(case, rng)
    if case["qkv"]:  # the projections come as column ranges of one matrix
        q, k, v = torch.randn((batch * slots, sum(widths)), generator=gen, device=DEV, dtype=dtype).split(widths, 1)
    else:
        q, k, v = (torch.randn((batch * slots, w), generator=gen, device=DEV, dtype=dtype) for w in widths)
    s = {"q": q, "k": k, "v": v, "table": _gpu(table), "ctx_len": _gpu(np.array(_lengths(batch, case["ctx"], 0), np.int32)),
         "k_cache": _cache(case, pages, gen, dtype), "v_cache": _cache(case, pages, gen, dtype), "pos": None, "rows": None}
    if slots <= 64:
        _, depth, mask = _trees(rng, batch, slots)
        s["pos"] = _gpu(depth)
        if case["accepted"]:  # the path to one slot of each tree, from the root down
            leaf = np.minimum(rng.integers(1, slots, batch), np.array(_valid(batch, slots)) - 1)
            path = np.full((batch, slots), -1, np.int32)
            for b in range(batch):
                on = [j for j in range(slots) if int(mask[b, leaf[b]]) >> j & 1]
                path[b, :len(on)] = on
            s["rows"] = _gpu(path)
    length = case["ctx"] + case["prefix"] + slots
    freq = 10000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"])
    angle = np.arange(length)[:, None] * freq
    s["rope"] = _gpu(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    s["q_out"] = torch.zeros((batch * slots, widths[0]), device=DEV, dtype=dtype)
    if own:
        s["kv"] = _kv_handle(case, pages)
    return s


def _prepare_attend(case, rng, gen):
    batch, slots, dim, dtype = case["batch"], case["slots"], case["dim"], TYPES[case["type"]]
    prefix_pages, table, pages = _cache_plan(case, rng)
    _, _, mask = _trees(rng, batch, slots)
    # queries of unit variance give scores of variance 1, flatter than trained heads: 2.5 times that
    q = torch.randn((batch * slots, case["q_heads"] * dim), generator=gen, device=DEV, dtype=dtype) * 2.5
    s = {"q": q, "k_cache": _cache(case, pages, gen, dtype), "v_cache": _cache(case, pages, gen, dtype),
         "table": _gpu(table), "prefix_pages": _gpu(prefix_pages) if case["prefix"] else None,
         "ctx_len": _gpu(np.array(_lengths(batch, case["ctx"], 0), np.int32)), "mask": _gpu(mask.view(np.int64)),
         "out": torch.zeros_like(q), "lse": torch.zeros((batch * slots, case["q_heads"]), device=DEV)}
    if own:
        s["kv"] = _kv_handle(case, pages)
    return s


def _prepare_logits(case, rng, gen):
    batch, slots, V, dtype = case["batch"], case["slots"], case["vocab"], TYPES[case["type"]]
    wide = torch.randn((batch * slots, V + case["pad"]), generator=gen, device=DEV, dtype=dtype)
    logits = wide[:, :V]
    active = rng.choice(V, min(V, 2000), replace=False)
    _, _, mask = _trees(rng, batch, slots)
    tok = active[np.minimum(rng.zipf(1.3, (batch, slots)) - 1, len(active) - 1)].astype(np.int32)
    tok[mask == 0] = -1
    # the target's favourite successor of each slot, five above the rest, sometimes a token seen before
    high = active[rng.integers(0, len(active), (batch * slots, 1))]
    logits.scatter_add_(1, _gpu(high), torch.full((batch * slots, 1), 5.0, device=DEV, dtype=dtype))
    hist = active[np.minimum(rng.zipf(1.2, (batch, case["hist"])) - 1, len(active) - 1)].astype(np.int32)
    hist_len = np.array(_lengths(batch, case["hist"], 1), np.int32)
    penalty = np.stack([rng.choice([1.0, 1.1, 1.3], batch), rng.choice([0.0, 0.2, 0.5], batch),
                        rng.choice([0.0, 0.4], batch)], 1).astype(np.float32)
    s = {"logits": logits, "tok": _gpu(tok), "mask": _gpu(mask.view(np.int64)), "hist": _gpu(hist),
         "hist_len": _gpu(hist_len), "prompt_len": _gpu(hist_len // 2), "penalty": _gpu(penalty),
         "out": torch.zeros((batch * slots, V + case["pad"]), device=DEV, dtype=dtype)[:, :V]}
    if case["bias"]:
        n = min(case["bias"], V)
        ids = np.stack([rng.choice(V, n, replace=False) for _ in range(batch)]).astype(np.int32)
        s["bias_tok"], s["bias_val"] = _gpu(ids), _gpu(rng.choice([-100.0, -2.0, 1.5, 4.0], (batch, n)).astype(np.float32))
    if case["grammar"]:
        words = -(-V // 32)
        table = rng.integers(0, 1 << 32, (case["grammar"], words), dtype=np.uint64).astype(np.uint32)
        table[0::3] &= (rng.random((len(table[0::3]), words)) < 0.02) * np.uint32(0xFFFFFFFF)  # few tokens allowed
        table[1::3] |= (rng.random((len(table[1::3]), words)) < 0.98) * np.uint32(0xFFFFFFFF)  # few tokens forbidden
        s["grammar"] = _gpu(table.view(np.int32))
        s["grammar_row"] = _gpu(rng.integers(-1, case["grammar"], (batch, slots)).astype(np.int32))
    if own:
        import hybrid_draft_tree_gb300 as g
        s["graft"] = g.Graft(g.graft_default_config(V, min(batch, 1000), g.GRAFT_MODE_STATIC,
                                                    g.GRAFT_F32 if case["type"] == "f32" else g.GRAFT_BF16))
    return s


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    make = {"append": _prepare_append, "attend": _prepare_attend, "logits": _prepare_logits}[case["op"]]
    return {**make(case, rng, gen), "case": case}


# --------------------------------------------------------------------------------------------------------- one pass
def _by_token(cache, case):
    """A view [pages, page, kv_heads, dim] of a cache of either layout."""
    return cache if case["layout"] == "token" else cache.transpose(1, 2)


def _rotate(x, cos, sin, case):
    """x: [tokens, heads, dim] in 32 bits; cos, sin: [tokens, 1, rot / 2]."""
    rot = case["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = r[..., :rot // 2], r[..., rot // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_append(s):
    case = s["case"]
    batch, slots, dim, page, half = case["batch"], case["slots"], case["dim"], case["page"], case["rot"] // 2
    index = torch.arange(slots, device=DEV).expand(batch, slots)
    depth = index if s["pos"] is None else s["pos"].long()
    base = s["ctx_len"].long()[:, None]
    every = torch.arange(batch, device=DEV)[:, None]

    def angles(position):
        cs = s["rope"][position.clamp(min=0)].reshape(batch * slots, 1, -1)
        return cs[..., :half], cs[..., half:]

    row = index if s["rows"] is None else s["rows"].long()
    live = (row >= 0) & (depth.gather(1, row.clamp(min=0)) >= 0)
    row = torch.where(live, row, row[:, :1])         # a pad repeats its tree's root, which changes nothing
    at = base + torch.where(live, index, 0)
    cos, sin = angles(base + depth.gather(1, row))
    source = (every * slots + row).reshape(-1)
    pages, offset = s["table"].long()[every, at // page].reshape(-1), (at % page).reshape(-1)
    k = _rotate(s["k"][source].float().view(batch * slots, -1, dim), cos, sin, case)
    _by_token(s["k_cache"], case)[pages, offset] = k.to(s["k"].dtype)
    _by_token(s["v_cache"], case)[pages, offset] = s["v"][source].view(batch * slots, -1, dim)
    if case["accepted"]:
        return s["k_cache"], s["v_cache"]
    q = _rotate(s["q"].float().reshape(batch * slots, -1, dim), *angles(base + depth), case)
    s["q_out"].copy_(torch.where((depth >= 0).view(-1, 1), q.flatten(1), 0.0))
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s):
    case = s["case"]
    batch, slots, prefix, page = case["batch"], case["slots"], case["prefix"], case["page"]
    hk, dim, group = case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    keys, rows = case["ctx"] + slots, slots * group
    # [kv head, request, slot and query head of the group, dim]
    q = s["q"].float().view(batch, slots, hk, group, dim).permute(2, 0, 1, 3, 4).reshape(hk, batch, rows, dim)
    at = torch.arange(keys, device=DEV)
    pages = s["table"].long()[:, at // page]
    k = _by_token(s["k_cache"], case)[pages, at % page].float().permute(2, 0, 1, 3)      # [hk, batch, keys, dim]
    v = _by_token(s["v_cache"], case)[pages, at % page].float().permute(2, 0, 1, 3)
    node = at - s["ctx_len"].long()[:, None]                                             # [batch, keys]: slot of a key
    bit = (s["mask"][:, :, None] >> node.clamp(0, slots - 1)[:, None, :]) & 1
    seen = (node < 0)[:, None, :] | ((node < slots)[:, None, :] & (bit == 1))
    live = s["mask"] != 0
    seen = (seen & live[:, :, None]).repeat_interleave(group, 1)                         # [batch, rows, keys]
    score = (q @ k.transpose(-1, -2)) / math.sqrt(dim)
    score = score.masked_fill(~seen, -math.inf)
    if prefix:
        at = torch.arange(prefix, device=DEV)
        pages = s["prefix_pages"].long()[at // page]
        pk = _by_token(s["k_cache"], case)[pages, at % page].float().transpose(0, 1)     # [hk, prefix, dim]
        pv = _by_token(s["v_cache"], case)[pages, at % page].float().transpose(0, 1)
        first = (q.flatten(1, 2) @ pk.transpose(-1, -2)).view(hk, batch, rows, prefix) / math.sqrt(dim)
        first = first.masked_fill(~live.repeat_interleave(group, 1)[..., None], -math.inf)
        score = torch.cat([first, score], -1)
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


def _plain_logits(s):
    case = s["case"]
    batch, slots, V = case["batch"], case["slots"], case["vocab"]
    at = torch.arange(case["hist"], device=DEV)
    held, prompt = at < s["hist_len"][:, None], at < s["prompt_len"][:, None]
    count = torch.zeros((batch, V), device=DEV).scatter_add_(1, s["hist"].long(), (held & ~prompt).float())
    old = torch.zeros((batch, V), device=DEV).scatter_add_(1, s["hist"].long(), (held & prompt).float())
    # a slot's path below the root is output too
    bit = ((s["mask"][:, :, None] >> torch.arange(slots, device=DEV)) & 1).float()
    bit[:, :, 0] = 0
    n = count[:, None, :].repeat(1, slots, 1)
    n.scatter_add_(2, s["tok"].long().clamp(min=0)[:, None, :].expand(batch, slots, slots), bit)
    rep, freq, pres = (s["penalty"][:, i].view(batch, 1, 1) for i in range(3))
    x = s["logits"].unflatten(0, (batch, slots)).float()
    x = torch.where((n > 0) | (old > 0)[:, None, :], torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * n - pres * (n > 0)
    if case["bias"]:
        x += torch.zeros((batch, V), device=DEV).scatter_(1, s["bias_tok"].long(), s["bias_val"])[:, None, :]
    if case["grammar"]:
        words = s["grammar"][s["grammar_row"].long().clamp(min=0)]
        bits = ((words[..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).flatten(2)[..., :V]
        x = x.masked_fill((bits == 0) & (s["grammar_row"] >= 0)[..., None], -math.inf)
    s["out"].copy_(torch.where((s["tok"] >= 0)[..., None], x, 0.0).flatten(0, 1))
    return s["out"]


def run(s):
    case = s["case"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "logits": _plain_logits}[case["op"]](s)
    batch, slots = case["batch"], case["slots"]
    if case["op"] == "append":
        with_q = not case["accepted"]
        s["kv"].append(batch, slots, s["q"] if with_q else None, s["k"], s["v"], s["rope"], s["table"], s["ctx_len"],
                       s["k_cache"], s["v_cache"], s["q_out"] if with_q else None, prefix_len=case["prefix"],
                       pos=s["pos"], rows=s["rows"])
        return (s["q_out"], s["k_cache"], s["v_cache"]) if with_q else (s["k_cache"], s["v_cache"])
    if case["op"] == "attend":
        s["kv"].attend(batch, slots, s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx_len"], case["ctx"], s["out"],
                       prefix_pages=s["prefix_pages"], prefix_len=case["prefix"], tree_mask=s["mask"], lse=s["lse"])
        return s["out"], s["lse"]
    s["graft"].process_logits(batch, slots, s["logits"], s["out"], tree_tok=s["tok"], tree_mask=s["mask"],
                              hist=s["hist"], hist_len=s["hist_len"], prompt_len=s["prompt_len"], penalty=s["penalty"],
                              bias_tok=s.get("bias_tok"), bias_val=s.get("bias_val"), grammar=s.get("grammar"),
                              grammar_row=s.get("grammar_row"))
    return s["out"]


# ------------------------------------------------------------------------------------------------- what a pass costs
def work(case):
    batch, slots = case["batch"], case["slots"]
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "logits":
        rows, V = sum(_valid(batch, slots)), case["vocab"]
        lists = sum(_lengths(batch, case["hist"], 1)) * 4 + batch * case["bias"] * 8 + case["grammar"] * V / 8
        # a division or product, two products' subtractions and an addition for each logit
        return {"bytes": rows * V * size * 2 + lists + batch * slots * 16, "flops": rows * V * 4}
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        tokens = sum(_valid(batch, slots)) if slots <= 64 else batch * slots
        if case["accepted"]:
            tokens = min(tokens, batch * 5)  # about five accepted nodes a request
        heads = 2 * hk + (0 if case["accepted"] else hq)
        rotated = heads - hk
        return {"bytes": tokens * (heads * dim * size * 2 + case["rot"] * 4 + 12), "flops": tokens * rotated * case["rot"] * 3}
    ctx, valid = _lengths(batch, case["ctx"], 0), _valid(batch, slots)
    keys = case["prefix"] + sum(ctx) + sum(valid)
    pairs = sum(n * (case["prefix"] + c) for n, c in zip(valid, ctx)) + sum(valid) * min(slots, 4)
    return {"bytes": keys * hk * dim * size * 2 + batch * slots * (hq * (dim * size * 2 + 4) + 8),
            "flops": 4 * pairs * hq * dim}


# ------------------------------------------------------------------------------------------- the definition in 64 bits
def _exact_append(s):
    case = s["case"]
    batch, slots, dim, page, rot = case["batch"], case["slots"], case["dim"], case["page"], case["rot"]
    ctx = s["ctx_len"].cpu().numpy().astype(np.int64)
    table = s["table"].cpu().numpy()
    depth = np.tile(np.arange(slots), (batch, 1)) if s["pos"] is None else s["pos"].cpu().numpy().astype(np.int64)
    rows = np.tile(np.arange(slots), (batch, 1)) if s["rows"] is None else s["rows"].cpu().numpy().astype(np.int64)
    rope = s["rope"].double()

    def turned(x, b, r):
        """The rows (b, r) of x as complex numbers, each turned by its position's angle."""
        x = x[_gpu(b * slots + r)].double().view(len(b), -1, dim).clone()
        cs = rope[_gpu(ctx[b] + depth[b, r])]
        turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None, :]
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    b, i = np.nonzero(rows >= 0)
    r = rows[b, i]
    keep = depth[b, r] >= 0
    b, i, r = b[keep], i[keep], r[keep]
    at = ctx[b] + i
    pages, offset = _gpu(table[b, at // page].astype(np.int64)), _gpu(at % page)
    caches = []
    for cache, new in ((s["k_cache"], turned(s["k"], b, r)), (s["v_cache"], s["v"][_gpu(b * slots + r)].double().view(len(b), -1, dim))):
        cache = cache.double()
        _by_token(cache, case)[pages, offset] = new
        caches.append(cache)
    if case["accepted"]:
        return tuple(caches)
    b, r = np.nonzero(depth >= 0)
    q = torch.zeros((batch * slots, case["q_heads"] * dim), device=DEV, dtype=torch.float64)
    q[_gpu(b * slots + r)] = turned(s["q"], b, r).flatten(1)
    return (q, *caches)


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
    k_all, v_all = (_by_token(s[name], case).flatten(0, 1) for name in ("k_cache", "v_cache"))
    q = s["q"].view(batch, slots, hk, group, dim)
    for b in range(batch):
        n = int(ctx[b]) + slots
        places = np.concatenate([shared, table[b].astype(np.int64).repeat(page)[:n] * page + np.arange(n) % page])
        seen = np.ones((slots, prefix + n), bool)
        seen[:, prefix + n - slots:] = (mask[b][:, None] >> np.arange(slots, dtype=np.uint64)) & np.uint64(1)
        k, v = k_all[_gpu(places)].double(), v_all[_gpu(places)].double()
        score = torch.einsum("shgd,nhd->hgsn", q[b].double(), k) * dim ** -0.5
        score.masked_fill_(~_gpu(seen), -math.inf)
        on = _gpu(np.nonzero(mask[b])[0])
        z = torch.logsumexp(score[:, :, on], -1)
        weight = torch.exp(score[:, :, on] - z[..., None])
        out[b, on] = torch.einsum("hgsn,nhd->shgd", weight, v)
        lse[b, on] = z.permute(2, 0, 1)
    return out.view(batch * slots, -1), lse.view(batch * slots, -1)


def _exact_logits(s):
    case = s["case"]
    batch, slots, V = case["batch"], case["slots"], case["vocab"]
    host = {name: s[name].cpu().numpy() for name in ("tok", "hist", "hist_len", "prompt_len", "penalty")}
    mask = s["mask"].cpu().numpy().view(np.uint64)
    out = torch.zeros((batch * slots, V + case["pad"]), device=DEV, dtype=torch.float64)[:, :V]
    rules = {name: s[name].cpu().numpy() for name in ("bias_tok", "bias_val", "grammar", "grammar_row") if name in s}
    allowed = None
    if case["grammar"]:
        allowed = np.unpackbits(rules["grammar"].view(np.uint8), axis=1, bitorder="little")[:, :V].astype(bool)
        allowed = _gpu(allowed)
    for b in range(batch):
        n, p = int(host["hist_len"][b]), int(host["prompt_len"][b])
        base = np.bincount(host["hist"][b, p:n], minlength=V)
        prompt = np.zeros(V, bool)
        prompt[host["hist"][b, :p]] = True
        live = np.nonzero(host["tok"][b] >= 0)[0]
        count = _gpu(np.repeat(base[None], len(live), 0))
        path = ((mask[b][live][:, None] >> np.arange(slots, dtype=np.uint64)) & np.uint64(1)).astype(bool)
        path[:, 0] = False
        where, which = np.nonzero(path)
        count.index_put_((_gpu(where), _gpu(host["tok"][b][which].astype(np.int64))),
                         torch.ones(len(where), device=DEV, dtype=torch.int64), accumulate=True)
        rep, freq, pres = (float(x) for x in host["penalty"][b])
        x = s["logits"][b * slots + _gpu(live)].double()
        seen = (count > 0) | _gpu(prompt)
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x) - freq * count - pres * (count > 0)
        if case["bias"]:
            x[:, _gpu(rules["bias_tok"][b].astype(np.int64))] += _gpu(rules["bias_val"][b].astype(np.float64))
        if allowed is not None:
            row = rules["grammar_row"][b][live].astype(np.int64)
            x.masked_fill_(~allowed[_gpu(np.maximum(row, 0))] & _gpu(row >= 0)[:, None], -math.inf)
        out[b * slots + _gpu(live)] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "logits": _exact_logits}[case["op"]](s)
