"""The paged-cache append, the tree attention and the logit rules against plain implementations in 64 bits.

Tolerances follow from the number formats: u = 2^-8 (bf16) or 2^-11 (f16) is the largest relative error of one rounding
to the type, e = 2^-24 that of an fp32 operation; each test adds up the roundings of its formula.
"""
import math
import time

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import hybrid_draft_tree_gb300 as g  # noqa: E402
from hybrid_draft_tree_gb300 import graft as gb  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
GDT = {"bf16": g.GRAFT_BF16, "f16": g.GRAFT_F16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
E = 2.0 ** -24


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.cuda.set_device(0)


def make_cache(gen, pages, hk, page, dim, dtype, layout):
    shape = (pages, hk, page, dim) if layout == "head" else (pages, page, hk, dim)
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def by_token(cache, layout):
    return cache.transpose(1, 2) if layout == "head" else cache


def random_trees(rng, batch, slots, pads=True):
    parent = np.full((batch, slots), -1, np.int64)
    depth = np.full((batch, slots), -1, np.int32)
    mask = np.zeros((batch, slots), np.uint64)
    for b in range(batch):
        valid = int(rng.integers(max(1, slots - 3), slots + 1)) if pads else slots
        depth[b, 0], mask[b, 0] = 0, 1
        for i in range(1, valid):
            p = int(rng.integers(max(0, i - 6), i))
            parent[b, i], depth[b, i] = p, depth[b, p] + 1
            mask[b, i] = int(mask[b, p]) | (1 << i)
    return parent, depth, mask


def tables(rng, batch, tokens, prefix, page):
    own, pre = -(-tokens // page), -(-prefix // page)
    total = batch * own + pre + 2
    order = rng.permutation(total)[:total - 2].astype(np.int32)
    return order[:pre], order[pre:].reshape(batch, own), total


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ---------------------------------------------------------------------------------------------------------- append
def append_reference(q, k, v, rope, depth, rows, ctx, table, prefix, page, hq, hk, dim, rot, inter):
    """{(b, i): (page, offset, key, value)} in 64 bits and {(b, i): query}; bound of the rotation's fp32 error."""
    batch, slots = depth.shape
    q, k, v, rope = (None if x is None else x.double().cpu().numpy() for x in (q, k, v, rope))
    a = slice(0, rot, 2) if inter else slice(0, rot // 2)
    b_ = slice(1, rot, 2) if inter else slice(rot // 2, rot)

    def turn(x, pos):
        x, y = x.copy(), x.copy()
        c, s = rope[pos, :rot // 2], rope[pos, rot // 2:]
        y[:, a] = x[:, a] * c - x[:, b_] * s
        y[:, b_] = x[:, b_] * c + x[:, a] * s
        size = np.zeros_like(x)
        size[:, a] = size[:, b_] = np.abs(x[:, a]) + np.abs(x[:, b_])
        return y, size

    places, queries = {}, {}
    for b in range(batch):
        for i in range(slots):
            if q is not None and depth[b, i] >= 0:
                queries[b, i] = turn(q[b * slots + i].reshape(hq, dim), prefix + ctx[b] + depth[b, i])
            r = rows[b, i]
            if r < 0 or depth[b, r] < 0:
                continue
            at = ctx[b] + i
            kk = turn(k[b * slots + r].reshape(hk, dim), prefix + ctx[b] + depth[b, r])
            places[b, i] = (table[b, at // page], at % page, kk, v[b * slots + r].reshape(hk, dim))
    return places, queries


@pytest.mark.parametrize("dtype,batch,slots,hq,hk,dim,page,layout,rot,inter,shift,with_q,with_rows", [
    ("bf16", 1, 1, 8, 2, 128, 16, "head", 128, 0, 0, True, False),
    ("bf16", 3, 61, 32, 8, 128, 64, "head", 128, 0, 0, True, False),
    ("f16", 4, 17, 10, 2, 64, 8, "token", 64, 0, 0, True, True),
    ("bf16", 2, 64, 4, 4, 128, 128, "token", 64, 1, 0, True, False),
    ("f16", 2, 9, 5, 1, 128, 32, "head", 128, 1, 8, True, False),
    ("bf16", 2, 9, 6, 2, 64, 16, "head", 48, 0, 0, True, True),      # rot / 2 no multiple of 8 elements
    ("bf16", 2, 5, 4, 2, 64, 16, "token", 6, 1, 0, True, False),
    ("bf16", 2, 5, 4, 2, 64, 16, "head", 0, 0, 0, True, False),      # nothing rotates
    ("f16", 3, 13, 8, 2, 128, 16, "head", 128, 0, 3, True, False),   # rows off 16-byte boundaries
    ("bf16", 3, 13, 8, 2, 128, 16, "head", 128, 1, 1, False, True),
    ("bf16", 1, 1000, 4, 2, 128, 16, "head", 128, 0, 0, True, False),  # a prefill
])
def test_append(dtype, batch, slots, hq, hk, dim, page, layout, rot, inter, shift, with_q, with_rows):
    rng = np.random.default_rng(slots * 7 + dim + rot)
    gen = torch.Generator(device="cuda").manual_seed(slots)
    dt = DT[dtype]
    ctx = rng.integers(0, 3 * page, batch).astype(np.int32)
    ctx[0] = 0
    prefix = int(rng.integers(0, 50))
    _, table, pages = tables(rng, batch, int(ctx.max()) + slots, 0, page)
    widths = [hq * dim, hk * dim, hk * dim]
    qkv = torch.randn((batch * slots, sum(widths) + shift), generator=gen, device="cuda", dtype=dt)[:, shift:]
    q, k, v = qkv.split(widths, 1)
    k_cache, v_cache = (make_cache(gen, pages, hk, page, dim, dt, layout) for _ in range(2))
    k0, v0 = k_cache.clone(), v_cache.clone()
    if slots <= 64:
        _, depth, _ = random_trees(rng, batch, slots)
        pos = cuda(depth)
    else:
        depth, pos = np.tile(np.arange(slots, dtype=np.int32), (batch, 1)), None
    rows = np.tile(np.arange(slots), (batch, 1))
    if with_rows:
        rows = rng.integers(-1, slots, (batch, slots))
    positions = prefix + int(ctx.max()) + slots
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    rope = cuda(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)) if rot else None
    q_out = torch.full((batch * slots, hq * dim + shift), 7.0, device="cuda", dtype=dt)[:, shift:] if with_q else None
    kv = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, min(slots, 64), GDT[dtype], layout=layout,
                                             rot_dim=rot, rot_interleaved=inter))
    kv.append(batch, slots, q if with_q else None, k, v, rope, cuda(table), cuda(ctx), k_cache, v_cache, q_out,
              prefix_len=prefix, pos=pos, rows=cuda(rows.astype(np.int32)) if with_rows else None)
    assert kv.sync() == 0 and kv.last_launch_count() == 1
    if rope is None:
        rope = torch.zeros((positions, 0), device="cuda")
    places, queries = append_reference(q if with_q else None, k, v, rope, depth, rows, ctx, table, prefix, page, hq, hk,
                                       dim, rot, inter)
    kt, vt = by_token(k_cache, layout).double().cpu().numpy(), by_token(v_cache, layout).double().cpu().numpy()
    want_k, want_v = by_token(k0, layout).double().cpu().numpy(), by_token(v0, layout).double().cpu().numpy()
    slack = np.zeros_like(want_k)
    # two products, a sum and the table's own fp32 entries: 3 e of |a| + |b|, then one rounding to the type
    for p, off, (y, size), val in places.values():
        want_k[p, off], want_v[p, off] = y, val
        slack[p, off] = U[dt] * np.abs(y) + 4 * E * size + TINY[dt]
    assert np.all(np.abs(kt - want_k) <= slack)
    assert np.array_equal(vt, want_v)
    if with_q:
        got = q_out.double().cpu().numpy().reshape(batch, slots, hq, dim)
        for b in range(batch):
            for i in range(slots):
                if (b, i) in queries:
                    y, size = queries[b, i]
                    assert np.all(np.abs(got[b, i] - y) <= U[dt] * np.abs(y) + 4 * E * size + TINY[dt]), (b, i)
                else:
                    assert np.all(got[b, i] == 7.0)


def test_append_in_place_queries_and_other_stream():
    rng, gen = np.random.default_rng(5), torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((12, w * 64), generator=gen, device="cuda", dtype=torch.bfloat16) for w in (4, 2, 2))
    rope = torch.rand((40, 64), generator=gen, device="cuda")
    _, table, pages = tables(rng, 2, 20, 0, 8)
    table, ctx = cuda(table), cuda(np.array([3, 9], np.int32))
    kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 8, pages, 2, 6))
    caches = [torch.zeros((pages, 2, 8, 64), device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    out = torch.zeros_like(q)
    kv.append(2, 6, q, k, v, rope, table, ctx, caches[0], caches[1], out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv.append(2, 6, q, k, v, rope, table, ctx, caches[2], caches[3], q, stream=side)
    side.synchronize()
    assert kv.sync() == 0
    assert torch.equal(q, out) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_append_bad_data_is_flagged_and_skipped():
    """A page outside the cache, a place beyond the table, a row outside the request, a position beyond the table of
    angles and a negative length: the write is skipped, the rest lands, the error word says so."""
    hk, dim, page = 2, 64, 8
    k = torch.ones((4 * 3, hk * dim), device="cuda", dtype=torch.bfloat16)
    rope = torch.zeros((16, dim), device="cuda")
    rope[:, :dim // 2] = 1.0
    table = cuda(np.array([[0, 1], [2, 99], [3, -1], [4, 5]], np.int32))
    kv = g.GraftKV(g.graft_kv_default_config(hk, hk, dim, page, 6, 4, 3))

    def one(ctx, rows=None, rope_=rope):
        kc, vc = (torch.zeros((6, hk, page, dim), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        kv.append(4, 3, None, k, k, rope_, table, cuda(np.array(ctx, np.int32)), kc, vc, None,
                  rows=None if rows is None else cuda(np.array(rows, np.int32)))
        flags = kv.sync(raise_on_error=False)
        assert torch.equal(kc, vc)
        return flags, (kc[:, 0, :, 0] == 1).sum(1).tolist()

    assert one([0, 0, 0, 0]) == (0, [3, 0, 3, 3, 3, 0])
    assert one([0, 6, 6, 0]) == (gb.GRAFT_ERR_RANGE, [3, 0, 2, 2, 3, 0])      # pages 99 and -1
    assert one([0, 0, 0, 15]) == (gb.GRAFT_ERR_RANGE, [3, 0, 3, 3, 0, 1])     # beyond two pages, and positions 16, 17
    assert one([0, 0, 0, -1]) == (gb.GRAFT_ERR_RANGE, [3, 0, 3, 3, 0, 0])
    assert one([0, 0, 0, 0], rows=[[0, 1, 3], [0, -1, -1], [2, 1, 0], [-5, -1, 0]]) == (gb.GRAFT_ERR_RANGE,
                                                                                    [2, 0, 1, 3, 1, 0])
    assert one([0, 0, 0, 0], rope_=rope[:2]) == (gb.GRAFT_ERR_RANGE, [2, 0, 2, 2, 2, 0])


# ---------------------------------------------------------------------------------------------------------- attend
def attend_reference(q, k_cache, v_cache, layout, pre, table, prefix, ctx, mask, page, hq, hk, dim, scale):
    """out, lse and the bounds' ingredients in 64 bits: the weighted sum of |v| and the largest sum |q k| of a row."""
    batch, slots = mask.shape
    group = hq // hk
    out = torch.zeros((batch, slots, hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((batch, slots, hq), -math.inf, dtype=torch.float64, device="cuda")
    spread, reach = torch.zeros_like(out), torch.zeros_like(lse)
    kt, vt = by_token(k_cache, layout), by_token(v_cache, layout)
    qd = q.double().view(batch, slots, hk, group, dim)
    for b in range(batch):
        for i in range(slots):
            if mask[b, i] == 0:
                continue
            places = [(pre[p // page], p % page) for p in range(prefix)]
            places += [(table[b, p // page], p % page) for p in range(ctx[b])]
            places += [(table[b, (ctx[b] + j) // page], (ctx[b] + j) % page) for j in range(slots) if int(mask[b, i]) >> j & 1]
            at = cuda(np.array(places, np.int64).T)
            k, v = kt[at[0], at[1]].double(), vt[at[0], at[1]].double()       # [n, hk, dim]
            s = torch.einsum("hgd,nhd->hgn", qd[b, i], k) * scale
            size = torch.einsum("hgd,nhd->hgn", qd[b, i].abs(), k.abs()).amax(-1) * scale
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - z[..., None])
            out[b, i] = torch.einsum("hgn,nhd->hgd", w, v).reshape(hq, dim)
            spread[b, i] = torch.einsum("hgn,nhd->hgd", w, v.abs()).reshape(hq, dim)
            lse[b, i], reach[b, i] = z.reshape(hq), size.reshape(hq)
    return out, lse, spread, reach


def check_attend(got, got_lse, ref, dt, keys):
    out, lse, spread, reach = ref
    dim = out.shape[-1]
    got = got.double().view(out.shape)
    # a score's fp32 sum of dim products, its scaling and the exponent's argument: (dim + 8) e of sum |q k|; a weight is
    # rounded to the type (u); sums over the keys and rescalings: keys e; the result is rounded to the type (u)
    weight = (dim + 8) * E * (reach + 16)
    slack = (U[dt] + 2 * weight[..., None] + (keys + 64) * E) * spread + U[dt] * out.abs() + TINY[dt] * 2
    finite = torch.isfinite(out)
    assert torch.equal(torch.isfinite(got), finite)
    assert torch.all(((got - out).abs() <= slack)[finite])
    if got_lse is not None:
        z = got_lse.double().view(lse.shape)
        empty = lse == -math.inf
        assert torch.equal(z == -math.inf, empty)
        assert torch.all(((z - lse).abs() <= weight + (keys + 16) * E + 2 * E * lse.abs())[~empty])


def run_attend(dtype, batch, slots, prefix, ctx, hq, hk, dim, page, layout, causal=False, shift=0, scale=None, seed=0,
               tweak=None, max_ctx=None, q_scale=2.0):
    rng = np.random.default_rng(seed + slots * 3 + prefix)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    dt = DT[dtype]
    ctx = np.array(ctx, np.int32)
    pre, table, pages = tables(rng, batch, int(max(ctx.max(), max_ctx or 0)) + slots, prefix, page)
    k_cache, v_cache = (make_cache(gen, pages, hk, page, dim, dt, layout) for _ in range(2))
    q = (torch.randn((batch * slots, hq * dim + shift), generator=gen, device="cuda", dtype=dt) * q_scale)[:, shift:]
    if causal:
        mask = np.array([[(1 << (i + 1)) - 1 for i in range(slots)]] * batch, np.uint64)
    else:
        _, _, mask = random_trees(rng, batch, slots)
    if tweak:
        tweak(rng, q, by_token(k_cache, layout), by_token(v_cache, layout), pre, table, ctx, mask, page)
    out = torch.full((batch * slots, hq * dim + shift), 3.0, device="cuda", dtype=dt)[:, shift:]
    lse = torch.full((batch * slots, hq), 3.0, device="cuda")
    kv = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, slots, GDT[dtype], layout=layout))
    kv.attend(batch, slots, q, k_cache, v_cache, cuda(table), cuda(ctx), int(ctx.max()) if max_ctx is None else max_ctx,
              out, prefix_pages=cuda(pre) if prefix else None, prefix_len=prefix,
              tree_mask=None if causal else cuda(mask.view(np.int64)), scale=scale, lse=lse)
    assert kv.sync() == 0
    ref = attend_reference(q, k_cache, v_cache, layout, pre, table, prefix, ctx, mask, page, hq, hk, dim,
                           dim ** -0.5 if scale is None else scale)
    check_attend(out, lse, ref, dt, prefix + int(ctx.max()) + slots)
    return out, lse, kv


ATTEND = [
    # dtype, batch, slots, prefix, ctx, hq, hk, dim, page, layout
    ("bf16", 1, 1, 0, [0], 1, 1, 128, 8, "head"),               # one key, the query's own
    ("bf16", 1, 1, 0, [117], 32, 8, 128, 16, "head"),
    ("bf16", 2, 1, 0, [127, 128], 8, 2, 128, 16, "head"),       # the slot opens or ends a block of 128 keys
    ("f16", 3, 2, 1, [0, 1, 129], 5, 1, 64, 16, "token"),
    ("bf16", 4, 17, 128, [1, 200, 0, 63], 40, 8, 64, 32, "head"),
    ("f16", 2, 61, 300, [64, 70], 8, 2, 128, 64, "head"),
    ("bf16", 2, 64, 129, [0, 128], 4, 4, 128, 128, "token"),    # group 1, 64 slots
    ("bf16", 3, 3, 1000, [5, 250, 0], 16, 1, 128, 8, "token"),  # group 16
    ("f16", 9, 5, 77, [9, 8, 7, 6, 5, 4, 3, 2, 1], 6, 2, 64, 128, "head"),
    ("bf16", 1, 61, 0, [3001], 8, 2, 128, 16, "head"),          # few rows, a long axis
    ("bf16", 1, 2, 2500, [600], 2, 2, 64, 64, "token"),
    ("bf16", 20, 1, 700, list(range(0, 600, 30)), 8, 2, 128, 16, "head"),
    ("f16", 1, 64, 0, [0], 96, 1, 128, 64, "head"),             # 6144 rows of one head
    ("bf16", 1, 3, 200, [150], 130, 1, 128, 16, "head"),        # a group of more than 128 query heads
    ("bf16", 2, 2, 0, [5, 140], 300, 2, 64, 32, "token"),
    ("f16", 500, 1, 140, [b % 37 for b in range(500)], 2, 1, 64, 16, "head"),   # more requests than a CTA has threads
    ("bf16", 3, 50, 260, [513, 40, 128], 21, 7, 128, 8, "token"),   # rows that fill no tile: 126 of 128
    # more items than SMs, cut: of one tile with small pages, of two tiles
    ("bf16", 60, 2, 0, [(37 * b) % 1900 for b in range(60)], 8, 4, 128, 32, "head"),
    ("bf16", 30, 61, 0, [(53 * b) % 900 for b in range(30)], 32, 8, 64, 64, "head"),
    ("f16", 24, 40, 0, [(71 * b) % 1300 for b in range(24)], 32, 8, 128, 16, "token"),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}-b{c[1]}-s{c[2]}-p{c[3]}-h{c[5]}x{c[6]}-d{c[7]}-g{c[8]}{c[9]}")
def test_attend(case):
    run_attend(*case)


@pytest.mark.parametrize("slots,ctx", [(1, 40), (64, 200), (33, 0)])
def test_attend_causal_without_a_mask(slots, ctx):
    run_attend("bf16", 2, slots, 40, [ctx, ctx // 2], 4, 2, 128, 16, "head", causal=True)


@pytest.mark.parametrize("shift", [1, 8])
def test_attend_rows_at_any_stride_and_offset(shift):
    run_attend("bf16", 2, 9, 30, [33, 250], 8, 2, 128, 16, "token", shift=shift)


def test_attend_scale_and_large_scores():
    """Scores in the hundreds: the running maximum keeps every exponent finite."""
    run_attend("bf16", 2, 5, 200, [300, 40], 8, 2, 128, 16, "head", scale=1.0, q_scale=6.0)
    run_attend("f16", 1, 1, 0, [1000], 4, 1, 64, 16, "head", scale=2.0)
    run_attend("bf16", 1, 7, 260, [150], 4, 1, 128, 16, "head", scale=1e-6)


def test_attend_rising_scores():
    """Keys whose scores rise along the cache, so that the maximum moves in every block of keys."""
    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        for b in range(len(ctx)):
            for at in range(int(ctx[b])):
                k[table[b, at // page], at % page] *= 0.02 + at / 400.0
    run_attend("bf16", 2, 4, 0, [1500, 900], 4, 2, 128, 64, "head", tweak=tweak)


@pytest.mark.parametrize("dtype,dim,slots,step", [("f16", 64, 4, 40), ("bf16", 64, 61, 130), ("f16", 128, 61, 130), ("bf16", 128, 1, 300)])
def test_attend_scores_that_run_away_again_and_again(dtype, dim, slots, step):
    """Scores that rise by about 2^20 every `step` keys: weights are computed, found too large and written again with the
    new base, in block after block; the result is the definition's, and the same each time."""
    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        q.zero_()
        q.view(slots, -1, dim)[..., :2] = 2.0
        for at in range(int(ctx[0])):
            k[table[0, at // page], at % page, :, 0] = 7.0 * (at // step)
    first = run_attend(dtype, 1, slots, 0, [1500], 4, 2, dim, 16, "head", scale=1.0, tweak=tweak)[0]
    for _ in range(3):
        assert torch.equal(first, run_attend(dtype, 1, slots, 0, [1500], 4, 2, dim, 16, "head", scale=1.0, tweak=tweak)[0])


@pytest.mark.parametrize("dim", [64, 128])
def test_attend_large_values_behind_a_late_maximum(dim):
    """Values of 1e25 whose keys outscore the first ones by 2^46: no intermediate sum leaves fp32."""
    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        q.zero_()
        q.view(len(ctx), -1, 4, dim)[..., 0] = 8.0
        k.zero_()
        k[..., 0] = 4.0
        for at in range(200):
            k[table[0, at // page], at % page] = 0.0
        v *= 1e25
    run_attend("bf16", 1, 3, 0, [700], 4, 2, dim, 64, "head", scale=1.0, tweak=tweak)


@pytest.mark.parametrize("dim", [64, 128])
def test_attend_values_at_the_stated_bound(dim):
    """704 keys of values up to 2^115 / 704, most of them 2^11.9 ahead of the first ones, which is as far as a base stays:
    the sums are finite."""
    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        q.zero_()
        q.view(len(ctx), -1, 4, dim)[..., 0] = 1.0
        k.zero_()
        k[..., 0] = 8.25
        for at in range(200):
            k[table[0, at // page], at % page] = 0.0
        v.clamp_(0.5, 1.0)
        v *= 2.0 ** 115 / 704
    run_attend("bf16", 1, 4, 0, [700], 4, 2, dim, 64, "head", scale=1.0, tweak=tweak)


def test_attend_ctx_bound_above_every_length():
    """max_ctx is a bound: lengths far below it, zero among them, leave whole splits of the key axis empty."""
    run_attend("bf16", 3, 3, 0, [0, 5, 300], 8, 2, 128, 16, "head", max_ctx=9000)
    run_attend("bf16", 3, 1, 500, [0, 5, 300], 8, 2, 128, 16, "head", max_ctx=9000)
    run_attend("f16", 2, 61, 90, [0, 129], 8, 2, 64, 16, "token", max_ctx=5000)


def test_attend_masks_that_leave_nothing():
    """Pads give zeros and -inf whatever the caches hold; a mask without the slot's own bit and no context is no pad."""
    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        mask[0, :] = 0
        mask[1, 2] = 1 << 1
        mask[1, 3] = 0
    out, lse, _ = run_attend("bf16", 2, 5, 0, [40, 0], 4, 2, 128, 16, "head", tweak=tweak)
    assert torch.all(out[:5] == 0) and torch.all(lse[:5] == -math.inf) and torch.all(out[8] == 0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dims", [(2, 9, 37, [130, 61]), (3, 1, 200, [20, 0, 100]), (1, 61, 0, [1000])])
def test_attend_what_is_not_seen_has_no_effect(value, dims):
    """Everything a request does not see is NaN or infinite: the rest of its pages, the prefix's last page after its
    end, the pads' slots, pages of nobody.  Pads' queries are too."""
    batch, slots, prefix, ctx = dims
    seen = {}

    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        keep = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
        for p in range(prefix):
            keep[pre[p // page], p % page] = True
        for b in range(batch):
            some = 0
            for i in range(slots):
                some |= int(mask[b, i])
                if mask[b, i] == 0:
                    q[b * slots + i] = value
            for at in range(int(ctx[b]) + slots):
                if at < ctx[b] or some >> (at - int(ctx[b])) & 1:
                    keep[table[b, at // page], at % page] = True
        k[~keep] = value
        v[~keep] = value
        seen["out"] = int((~keep).sum())
    run_attend("bf16", batch, slots, prefix, ctx, 8, 2, 128, 16, "head", tweak=tweak)
    assert seen["out"] > 0


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attend_non_finite_slots_reach_only_those_that_see_them(value):
    """A slot whose key or value is not finite spoils its own subtree and nothing else."""
    rng = np.random.default_rng(0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    batch, slots, ctx, page = 2, 40, np.array([100, 7], np.int32), 16
    _, table, pages = tables(rng, batch, 140, 0, page)
    _, _, mask = random_trees(rng, batch, slots, pads=False)
    k, v = (make_cache(gen, pages, 2, page, 128, torch.bfloat16, "head") for _ in range(2))
    q = torch.randn((batch * slots, 8 * 128), generator=gen, device="cuda", dtype=torch.bfloat16)
    kv = g.GraftKV(g.graft_kv_default_config(8, 2, 128, page, pages, batch, slots))

    def attend():
        out = torch.empty_like(q)
        kv.attend(batch, slots, q, k, v, cuda(table), cuda(ctx), 100, out, tree_mask=cuda(mask.view(np.int64)))
        assert kv.sync() == 0
        return out.view(batch, slots, 8, 128)

    clean = attend()
    bad = {(0, 5): v, (0, 17): v, (1, 30): v, (1, 11): k}
    for (b, j), cache in bad.items():
        at = int(ctx[b]) + j
        if cache is v:
            cache[table[b, at // page], 0, at % page, 3] = value     # kv head 0, one element
        else:
            cache[table[b, at // page], 0, at % page] = value
    out = attend()
    for b in range(batch):
        for i in range(slots):
            sees_v = any((b == x and c is v and int(mask[b, i]) >> j & 1) for (x, j), c in bad.items())
            sees_k = any((b == x and c is k and int(mask[b, i]) >> j & 1) for (x, j), c in bad.items())
            assert torch.equal(out[b, i, 4:], clean[b, i, 4:])           # heads of kv head 1
            rest = [d for d in range(128) if d != 3]
            if not sees_k:
                # dropping and adding an element apart moves nothing else
                assert torch.equal(out[b, i, :4][:, rest], clean[b, i, :4][:, rest]), (b, i)
                assert torch.isfinite(out[b, i, :4, 3]).all() == (not sees_v), (b, i)
                if not sees_v:
                    assert torch.equal(out[b, i, :4, 3], clean[b, i, :4, 3])
            elif value != value:
                assert not torch.isfinite(out[b, i, :4]).any()


CLEANED = [
    # dtype, batch, slots, prefix, ctx, hq, hk, dim, page, layout
    ("f16", 2, 9, 37, [130, 61], 8, 2, 64, 8, "token"),
    ("f16", 2, 61, 300, [64, 70], 8, 2, 128, 128, "head"),
    ("bf16", 3, 1, 200, [20, 0, 100], 8, 2, 64, 128, "head"),
    ("f16", 1, 61, 0, [3001], 8, 2, 64, 16, "head"),                # cut and joined, two copying warps
    ("bf16", 1, 61, 0, [3001], 32, 2, 128, 8, "token"),             # of two tiles
    ("f16", 20, 3, 700, list(range(0, 600, 30)), 8, 2, 128, 32, "head"),   # packed
    ("bf16", 30, 61, 0, [(53 * b) % 900 for b in range(30)], 32, 8, 64, 8, "head"),   # more items than SMs
]


@pytest.mark.parametrize("value", [float("nan"), -float("inf")])
@pytest.mark.parametrize("case", CLEANED, ids=lambda c: f"{c[0]}-b{c[1]}-s{c[2]}-p{c[3]}-d{c[7]}-g{c[8]}{c[9]}")
def test_attend_cleans_values_in_every_form(case, value):
    """Each type, head and page size, item whole, cut, packed: what nobody sees is not finite, and so are a few elements of
    some slots' values, which reach the rows that see them and no others."""
    batch, slots, prefix, ctx = case[1:5]
    spoiled = []

    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        keep = torch.zeros(k.shape[:2], dtype=torch.bool)
        for p in range(prefix):
            keep[pre[p // page], p % page] = True
        for b in range(batch):
            for at in range(int(ctx[b]) + slots):
                seen = at < ctx[b] or any(int(m) >> (at - int(ctx[b])) & 1 for m in mask[b])
                keep[table[b, at // page], at % page] = bool(seen)
        keep = keep.cuda()
        k[~keep] = value
        v[~keep] = value
        for b in range(0, batch, 2):
            for j in {slots // 3, slots - 1}:
                if mask[b, j]:
                    at = int(ctx[b]) + j
                    v[table[b, at // page], at % page, 0, 5] = value
                    v[table[b, at // page], at % page, -1, -1] = value
                    spoiled.append((b, j))
    out, _, _ = run_attend(*case, tweak=tweak)
    assert spoiled and not torch.isfinite(out).all()


def test_attend_finite_slots_are_untouched_by_cleaning():
    """The largest numbers of each type, subnormal ones and both zeros in slots' values are no infinities."""
    for dtype, dim in (("f16", 64), ("f16", 128), ("bf16", 64)):
        top = torch.finfo(DT[dtype]).max if dtype == "f16" else 1e30

        def tweak(rng, q, k, v, pre, table, ctx, mask, page):
            for j, x in enumerate((top, -top, torch.finfo(DT[dtype]).tiny / 4, -0.0)):
                at = int(ctx[0]) + j
                v[table[0, at // page], at % page, :, j::7] = x
        run_attend(dtype, 1, 9, 0, [125], 4, 2, dim, 16, "head", tweak=tweak)


def test_attend_bad_data_is_flagged_and_stays_in_bounds():
    rng, gen = np.random.default_rng(1), torch.Generator(device="cuda").manual_seed(1)
    k, v = (make_cache(gen, 8, 2, 16, 64, torch.bfloat16, "head") for _ in range(2))
    q = torch.randn((2, 4 * 64), generator=gen, device="cuda", dtype=torch.bfloat16)
    kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 16, 8, 2, 1))
    out = torch.empty_like(q)

    def flags(table, ctx, pre=None, n=0):
        kv.attend(2, 1, q, k, v, cuda(np.array(table, np.int32)), cuda(np.array(ctx, np.int32)), 40, out,
                  prefix_pages=None if pre is None else cuda(np.array(pre, np.int32)), prefix_len=n)
        return kv.sync(raise_on_error=False)

    good = [[0, 1, 2], [3, 4, 5]]
    assert flags(good, [40, 10]) == 0
    assert flags([[0, 1, 2], [3, 400, -7]], [40, 10]) == 0          # pages that hold nothing yet
    assert flags([[0, 8, 2], [3, 4, 5]], [40, 10]) == gb.GRAFT_ERR_RANGE
    assert flags([[0, 1, 2], [-1, 4, 5]], [40, 10]) == gb.GRAFT_ERR_RANGE
    assert flags(good, [41, 10]) == gb.GRAFT_ERR_RANGE
    assert flags(good, [40, -1]) == gb.GRAFT_ERR_RANGE
    assert flags(good, [40, 10], [6, 1 << 30], 20) == gb.GRAFT_ERR_RANGE
    assert flags(good, [40, 10], [6, 7], 20) == 0
    with pytest.raises(g.GraftError, match="range 1"):
        kv.attend(2, 1, q, k, v, cuda(np.array([[0, 8, 2], [3, 4, 5]], np.int32)), cuda(np.array([40, 10], np.int32)),
                  40, out)
        kv.sync()


def test_attend_repeats_bit_for_bit_and_from_a_graph_and_another_stream():
    out, lse, kv = run_attend("bf16", 5, 17, 900, [100, 0, 333, 64, 7], 8, 2, 128, 16, "head")
    again, again_lse, _ = run_attend("bf16", 5, 17, 900, [100, 0, 333, 64, 7], 8, 2, 128, 16, "head")
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    rng, gen = np.random.default_rng(2), torch.Generator(device="cuda").manual_seed(2)
    pre, table, pages = tables(rng, 3, 2001, 300, 16)
    k, v = (make_cache(gen, pages, 2, 16, 128, torch.bfloat16, "head") for _ in range(2))
    q = torch.randn((3, 8 * 128), generator=gen, device="cuda", dtype=torch.bfloat16)
    kv = g.GraftKV(g.graft_kv_default_config(8, 2, 128, 16, pages, 3, 1))
    table, pre, ctx = cuda(table), cuda(pre), cuda(np.array([2000, 1, 700], np.int32))
    outs = [torch.zeros_like(q) for _ in range(3)]
    call = lambda o, **s: kv.attend(3, 1, q, k, v, table, ctx, 2000, o, prefix_pages=pre, prefix_len=300, **s)  # noqa: E731
    call(outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(outs[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[2])
    graph.replay()
    ctx.copy_(torch.tensor([2000, 1, 700], dtype=torch.int32))
    graph.replay()
    assert kv.sync() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_attend_waits_are_bounded():
    """With a limit of one poll the kernel's waits run out: the call ends, says so, and the handle works on."""
    rng, gen = np.random.default_rng(4), torch.Generator(device="cuda").manual_seed(4)
    pre, table, pages = tables(rng, 3, 700, 300, 16)
    k, v = (make_cache(gen, pages, 2, 16, 128, torch.bfloat16, "head") for _ in range(2))
    kv = g.GraftKV(g.graft_kv_default_config(8, 2, 128, 16, pages, 3, 40))
    table, pre, ctx = cuda(table), cuda(pre), cuda(np.array([600, 1, 300], np.int32))
    for slots in (1, 40):
        q = torch.randn((3 * slots, 8 * 128), generator=gen, device="cuda", dtype=torch.bfloat16)
        outs = [torch.zeros_like(q) for _ in range(2)]
        call = lambda o: kv.attend(3, slots, q, k, v, table, ctx, 600, o, prefix_pages=pre, prefix_len=300)  # noqa: E731
        call(outs[0])
        assert kv.sync() == 0
        kv.set_wait_limit(1)
        call(outs[1])
        assert kv.sync(raise_on_error=False) == gb.GRAFT_ERR_TIMEOUT
        with pytest.raises(g.GraftError, match="timeout 1"):
            call(outs[1])
            kv.sync()
        kv.set_wait_limit(0)
        outs[1].zero_()
        call(outs[1])
        assert kv.sync() == 0
        assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("dim,page,ctx", [(128, 16, [600, 1, 300]), (64, 8, [600, 1, 300]), (128, 32, [9000]), (64, 16, [9000])])
def test_attend_bounded_waits_with_two_copying_warps(dim, page, ctx):
    """Small pages and one tile an item take two copying warps, which give up apart: the call ends at once all the same (a
    drain that waits for what was never asked for takes a second), says so, and the handle works on."""
    rng, gen = np.random.default_rng(6), torch.Generator(device="cuda").manual_seed(6)
    batch = len(ctx)
    _, table, pages = tables(rng, batch, max(ctx) + 1, 0, page)
    k, v = (make_cache(gen, pages, 2, page, dim, torch.bfloat16, "head") for _ in range(2))
    kv = g.GraftKV(g.graft_kv_default_config(8, 2, dim, page, pages, batch, 1))
    table, at = cuda(table), cuda(np.array(ctx, np.int32))
    q = torch.randn((batch, 8 * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    want, out = torch.zeros_like(q), torch.zeros_like(q)
    kv.attend(batch, 1, q, k, v, table, at, max(ctx), want)
    assert kv.sync() == 0
    expired = 0
    for limit in [1, 2, 3] * 20:
        kv.set_wait_limit(limit)
        start = time.perf_counter()
        kv.attend(batch, 1, q, k, v, table, at, max(ctx), out)
        flags = kv.sync(raise_on_error=False)
        assert time.perf_counter() - start < 0.5
        assert flags in (0, gb.GRAFT_ERR_TIMEOUT)
        assert flags or torch.equal(out, want)
        expired += flags != 0
    assert expired
    kv.set_wait_limit(0)
    out.zero_()
    kv.attend(batch, 1, q, k, v, table, at, max(ctx), out)
    assert kv.sync() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("order", [(1, 0, 2), (2, 0, 1), (2, 1, 0), (1, 2, 0)])
def test_strides_in_any_order(order):
    """Caches whose pages, heads and tokens nest in another order than pages first: `order` from the outermost in, of page
    (0), head (1), token (2)."""
    rng, gen = np.random.default_rng(3), torch.Generator(device="cuda").manual_seed(3)
    batch, slots, hq, hk, dim, page = 2, 5, 4, 2, 64, 16
    ctx = np.array([140, 33], np.int32)
    _, table, pages = tables(rng, batch, int(ctx.max()) + slots, 0, page)
    sizes = [pages, hk, page]
    k_all, v_all = (torch.randn([*[sizes[a] for a in order], dim], generator=gen, device="cuda", dtype=torch.bfloat16)
                    for _ in range(2))
    back = [order.index(a) for a in range(3)] + [3]
    k_cache, v_cache = k_all.permute(back), v_all.permute(back)                  # [page, head, token, dim]
    stride = k_cache.stride()
    kv = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, slots, page_stride=stride[0],
                                             head_stride=stride[1], token_stride=stride[2]))
    q, k, v = (torch.randn((batch * slots, h * dim), generator=gen, device="cuda", dtype=torch.bfloat16) for h in (hq, hk, hk))
    rope = torch.zeros((200, dim), device="cuda")
    rope[:, :dim // 2] = 1.0
    want_k, want_v = k_cache.clone(), v_cache.clone()
    for b in range(batch):
        for i in range(slots):
            at = int(ctx[b]) + i
            want_k[table[b, at // page], :, at % page] = k[b * slots + i].view(hk, dim)
            want_v[table[b, at // page], :, at % page] = v[b * slots + i].view(hk, dim)
    out, lse = torch.empty_like(q), torch.empty((batch * slots, hq), device="cuda")
    kv.append(batch, slots, None, k, v, rope, cuda(table), cuda(ctx), k_all, v_all, None)
    kv.attend(batch, slots, q, k_all, v_all, cuda(table), cuda(ctx), 140, out, lse=lse)
    assert kv.sync() == 0
    assert torch.equal(k_cache, want_k) and torch.equal(v_cache, want_v)
    mask = np.array([[(1 << (i + 1)) - 1 for i in range(slots)]] * batch, np.uint64)
    ref = attend_reference(q, want_k, want_v, "head", None, table, 0, ctx, mask, page, hq, hk, dim, dim ** -0.5)
    check_attend(out, lse, ref, torch.bfloat16, 145)


def test_offsets_beyond_32_bits():
    """Pages far apart in a cache of 2^31 elements and more: append writes and attend reads the right ones."""
    hk, dim, page, pages = 2, 128, 16, 5
    stride = (1 << 29) + 4096                                        # the last page starts beyond 2^31 elements
    cache = torch.zeros((pages - 1) * stride + hk * page * dim, device="cuda", dtype=torch.bfloat16)
    kv = g.GraftKV(g.graft_kv_default_config(4, hk, dim, page, pages, 1, 4, page_stride=stride))
    gen = torch.Generator(device="cuda").manual_seed(9)
    k = torch.randn((36, hk * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    rope = torch.zeros((64, dim), device="cuda")
    rope[:, :dim // 2] = 1.0
    table = cuda(np.array([[4, 3, 4 - 3]], np.int32))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.append(1, 36, None, k, k, rope, table, zero, cache, cache, None)
    assert kv.sync() == 0
    for n, p in ((0, 4), (16, 3), (32, 1)):
        rows = min(16, 36 - n)
        got = cache[p * stride:p * stride + hk * page * dim].view(hk, page, dim)[:, :rows].transpose(0, 1)
        assert torch.equal(got.reshape(rows, -1), k[n:n + rows])
    q = torch.randn((4, 4 * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((4, 4), device="cuda")
    kv.attend(1, 4, q, cache, cache, table, zero + 32, 32, out, lse=lse)
    assert kv.sync() == 0
    small = torch.zeros((3, hk, page, dim), device="cuda", dtype=torch.bfloat16)
    for n in range(36):
        small[n // 16, :, n % 16] = k[n].view(hk, dim)
    mask = np.array([[1, 3, 7, 15]], np.uint64)
    ref = attend_reference(q, small, small, "head", None, np.array([[0, 1, 2]]), 0, np.array([32]), mask, 16, 4, 2, dim,
                           dim ** -0.5)
    check_attend(out, lse, ref, torch.bfloat16, 36)


# ---------------------------------------------------------------------------------------------------------- logits
def logits_reference(x, V, slots, tok, mask, hist, hist_len, prompt_len, penalty, bias_tok, bias_val, grammar, gram_row):
    """(values, sizes) in 64 bits by loops over the rules; a row of pads is None."""
    rows = []
    for row in range(x.shape[0]):
        b, i = divmod(row, slots)
        if tok is not None and tok[b, i] < 0:
            rows.append(None)
            continue
        y = x[row].astype(np.float64).copy()
        n, prompt = np.zeros(V, np.int64), np.zeros(V, bool)
        if hist is not None:
            p = 0 if prompt_len is None else min(prompt_len[b], hist_len[b])
            prompt[hist[b, :p]] = True
            np.add.at(n, hist[b, p:hist_len[b]], 1)
        if tok is not None:
            for j in range(1, slots):
                if int(mask[b, i]) >> j & 1:
                    n[tok[b, j]] += 1
        r, f, p = (1.0, 0.0, 0.0) if penalty is None else (float(t) for t in penalty[b])
        seen = (n > 0) | prompt
        y = np.where(seen, np.where(y > 0, y / r, y * r), y)
        size = np.abs(y) + abs(f) * n + abs(p) * (n > 0)
        y = y - f * n - p * (n > 0)
        if bias_tok is not None:
            entry = {int(t): float(w) for t, w in zip(bias_tok[b], bias_val[b]) if t >= 0}
            for t, w in entry.items():
                y[t] += w
                size[t] += abs(w)
        if grammar is not None and gram_row[b, i] >= 0:
            words = grammar[gram_row[b, i]].view(np.uint32)
            allowed = (words[np.arange(V) >> 5] >> (np.arange(V) & 31).astype(np.uint32)) & 1
            y[allowed == 0] = -np.inf
        rows.append((y, size))
    return rows


LOGITS = [
    # dtype, batch, slots, V, hist, bias, grammar rows, offset of the rows, out's offset
    ("f32", 1, 1, 1, 3, 1, 1, 0, 0),
    ("f32", 1, 1, 32000, 300, 64, 2, 0, 0),
    ("bf16", 2, 61, 1003, 50, 5, 3, 0, 0),         # odd rows: each starts at another offset
    ("bf16", 3, 17, 40000, 4000, 300, 8, 0, 0),
    ("bf16", 2, 5, 9001, 700, 10, 2, 3, 3),
    ("bf16", 2, 5, 9001, 700, 10, 2, 3, 4),        # rows of input and output at different offsets
    ("f32", 2, 64, 5003, 100, 2046, 1, 1, 1),
    ("f32", 2, 3, 4099, 100, 0, 0, 2, 0),
    ("bf16", 1, 61, 128256, 0, 0, 4, 0, 0),
    ("bf16", 5, 1, 4097, 30000, 7, 5, 0, 0),       # a long history, one slot
    ("bf16", 1, 2, 31, 5, 3, 2, 0, 0),
    ("bf16", 32, 33, 40009, 60, 9, 3, 0, 0),       # many rows and chunks enough for all SMs, odd rows
    ("f32", 32, 32, 20012, 60, 9, 3, 0, 0),
    ("bf16", 40, 1, 50001, 9000, 5, 3, 0, 0),      # long histories, chunks enough to grow
]


def logits_inputs(dtype, batch, slots, V, hist, n_bias, n_gram, shift, out_shift, seed=0):
    rng = np.random.default_rng(seed + V + slots)
    gen = torch.Generator(device="cuda").manual_seed(V)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.randn((batch * slots, V + shift), generator=gen, device="cuda", dtype=dt)[:, shift:] * 3
    wide = torch.empty((batch * slots, V + shift), device="cuda", dtype=dt)
    wide[:, shift:] = x
    x = wide[:, shift:]
    few = rng.integers(0, V, 40)
    _, _, mask = random_trees(rng, batch, slots)
    tok = few[rng.integers(0, 40, (batch, slots))].astype(np.int32)
    tok[mask == 0] = -1
    s = dict(tok=tok, mask=mask, hist=None, hist_len=None, prompt_len=None, bias_tok=None, bias_val=None, grammar=None,
             gram_row=None)
    s["penalty"] = np.stack([rng.choice([0.8, 1.0, 1.3], batch), rng.choice([-0.3, 0.0, 0.7], batch),
                             rng.choice([0.0, 0.6], batch)], 1).astype(np.float32)
    if hist:
        s["hist"] = np.where(rng.random((batch, hist)) < 0.5, few[rng.integers(0, 40, (batch, hist))],
                             rng.integers(0, V, (batch, hist))).astype(np.int32)
        s["hist_len"] = rng.integers(0, hist + 1, batch).astype(np.int32)
        s["hist_len"][0] = hist
        s["prompt_len"] = rng.integers(0, hist + 1, batch).astype(np.int32)
    if n_bias:
        s["bias_tok"] = rng.integers(-1, V, (batch, n_bias)).astype(np.int32)   # repeats and empty entries among them
        s["bias_val"] = rng.normal(0, 5, (batch, n_bias)).astype(np.float32)
    if n_gram:
        words = (V + 31) // 32 + 1
        s["grammar"] = rng.integers(0, 1 << 32, (n_gram, words), dtype=np.uint64).astype(np.uint32)
        s["grammar"][0] = 0                                                     # allows nothing
        s["gram_row"] = rng.integers(-1, n_gram, (batch, slots)).astype(np.int32)
        s["gram_row"][0, 0] = 0
    out = torch.full((batch * slots, V + out_shift), 9.0, device="cuda", dtype=dt)[:, out_shift:]
    return x, out, s, dt


def call_logits(eng, batch, slots, x, out, s, **more):
    dev = {k: None if v is None else cuda(v.view(np.int32) if v.dtype == np.uint32 else v.view(np.int64)
                                          if v.dtype == np.uint64 else v) for k, v in s.items()}
    eng.process_logits(batch, slots, x, out, tree_tok=dev["tok"], tree_mask=dev["mask"], hist=dev["hist"],
                       hist_len=dev["hist_len"], prompt_len=dev["prompt_len"], penalty=dev["penalty"],
                       bias_tok=dev["bias_tok"], bias_val=dev["bias_val"], grammar=dev["grammar"],
                       grammar_row=dev["gram_row"], **more)


def check_logits(out, x_host, s, dt, V, slots, pad_value=9.0):
    got = out.double().cpu().numpy()
    want = logits_reference(x_host, V, slots, **s)
    for row, w in enumerate(want):
        if w is None:
            assert np.all(got[row] == pad_value)
            continue
        y, size = w
        fine = np.isfinite(y)
        assert np.array_equal(np.isnan(y), np.isnan(got[row])) and np.array_equal(np.isfinite(got[row]), fine)
        assert np.array_equal(got[row][~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)])
        # a quotient or product, f n, two differences and a sum: 6 e of the terms' sizes, then one rounding to the type
        slack = 6 * E * size + U[dt] * np.abs(y)
        assert np.all(np.abs(got[row] - y)[fine] <= slack[fine])


@pytest.mark.parametrize("case", LOGITS, ids=lambda c: "-".join(map(str, c)))
def test_process_logits(case):
    dtype, batch, slots, V = case[:4]
    x, out, s, dt = logits_inputs(*case)
    eng = g.Graft(g.graft_default_config(V, batch, g.GRAFT_MODE_STATIC, g.GRAFT_F32 if dtype == "f32" else g.GRAFT_BF16))
    host = x.double().cpu().numpy()
    call_logits(eng, batch, slots, x, out, s)
    assert eng.sync() == 0 and eng.last_launch_count() == 1
    check_logits(out, host, s, dt, V, slots)
    assert torch.equal(x.double().cpu(), torch.from_numpy(host))               # the input stays
    call_logits(eng, batch, slots, x, x, s)                                    # in place
    assert eng.sync() == 0
    pads = np.repeat(s["tok"].reshape(-1)[:, None] < 0, V, 1)
    assert torch.equal(torch.where(cuda(pads), out, x), out)
    eng.close()


@pytest.mark.parametrize("off", ["tree", "penalty", "bias", "grammar", "history"])
def test_process_logits_rules_that_are_off(off):
    case = ("bf16", 2, 9, 3001, 200, 20, 4, 0, 0)
    x, out, s, dt = logits_inputs(*case)
    for k in {"tree": ["tok", "mask"], "penalty": ["penalty"], "bias": ["bias_tok", "bias_val"],
              "grammar": ["grammar", "gram_row"], "history": ["hist", "hist_len", "prompt_len"]}[off]:
        s[k] = None
    eng = g.Graft(g.graft_default_config(3001, 2, g.GRAFT_MODE_STATIC, g.GRAFT_BF16))
    call_logits(eng, 2, 9, x, out, s)
    assert eng.sync() == 0
    check_logits(out, x.double().cpu().numpy(), s, dt, 3001, 9)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_process_logits_infinities_and_nan(dtype):
    case = (dtype, 2, 6, 700, 300, 30, 3, 0, 0)
    x, out, s, dt = logits_inputs(*case)
    s["penalty"][:] = [[1.2, 0.5, 0.1], [0.9, -0.5, 0.0]]
    x[:, 0::7] = float("inf")
    x[:, 1::7] = -float("inf")
    x[:, 2::7] = float("nan")
    x[:, 3::7] = torch.finfo(dt).min
    host = x.double().cpu().numpy()
    eng = g.Graft(g.graft_default_config(700, 2, g.GRAFT_MODE_STATIC, g.GRAFT_F32 if dtype == "f32" else g.GRAFT_BF16))
    call_logits(eng, 2, 6, x, out, s)
    assert eng.sync() == 0
    got = out.double().cpu().numpy()
    lowest = np.zeros(700, bool)
    lowest[3::7] = True
    for row, w in enumerate(logits_reference(host, 700, 6, **s)):
        if w is None:
            continue
        y, size = w
        # the type's lowest value times a penalty above 1 leaves the type's range
        y = np.where(lowest & (y < float(torch.finfo(dt).min)), -np.inf, y)
        fine = np.isfinite(y) & ~lowest
        assert np.array_equal(np.isnan(got[row]), np.isnan(y))
        assert np.array_equal(got[row][~fine & ~np.isnan(y) & ~lowest], y[~fine & ~np.isnan(y) & ~lowest])
        assert np.all(np.abs(got[row] - y)[fine] <= (6 * E * size + U[dt] * np.abs(y))[fine])
        low = got[row][lowest]
        ref = y[lowest]
        assert np.array_equal(np.isneginf(low)[np.isneginf(ref)], np.ones(np.isneginf(ref).sum(), bool))
        keep = np.isfinite(low)
        assert np.all(np.abs(low / ref - 1)[keep] <= 2 * U[dt])


def _ruled(V, batch, slots, bias, r=1.2, f=0.5, p=0.1):
    """Rules whose tokens are known: a chain of slots, prompt 20-22, output 30, 31, 31, 31, 5; `bias`: token -> value."""
    s = dict(tok=np.tile(np.arange(5, 5 + slots, dtype=np.int32), (batch, 1)),
             mask=np.array([[(1 << (i + 1)) - 1 for i in range(slots)]] * batch, np.uint64),
             hist=np.tile(np.array([20, 21, 22, 30, 31, 31, 31, 5], np.int32), (batch, 1)),
             hist_len=np.full(batch, 8, np.int32), prompt_len=np.full(batch, 3, np.int32),
             penalty=np.tile(np.array([r, f, p], np.float32), (batch, 1)), bias_tok=None, bias_val=None, grammar=None,
             gram_row=None)
    if bias:
        s["bias_tok"] = np.tile(np.array(list(bias), np.int32), (batch, 1))
        s["bias_val"] = np.tile(np.array(list(bias.values()), np.float32), (batch, 1))
    return s


def _run_logits(dtype, V, batch, slots, s, x):
    """The rules on x, out of place and then in place: both have to agree."""
    eng = g.Graft(g.graft_default_config(V, batch, g.GRAFT_MODE_STATIC, g.GRAFT_F32 if dtype == "f32" else g.GRAFT_BF16))
    out = torch.full_like(x, 9.0)
    call_logits(eng, batch, slots, x, out, s)
    y = x.clone()
    call_logits(eng, batch, slots, y, y, s)
    assert eng.sync() == 0
    eng.close()
    assert torch.equal(torch.where(torch.isnan(out), 0, out), torch.where(torch.isnan(y), 0, y))
    assert torch.equal(torch.isnan(out), torch.isnan(y))
    return out


@pytest.mark.parametrize("rules", [(1.2, 0.5, 0.1), (1.3, 0.0, 0.0), (1.0, 0.0, 0.0)])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_process_logits_infinite_biases(dtype, value, rules):
    """A bias of -inf bans its token, one of +inf forces it, wherever the token has occurred: in the output (31), the
    prompt (20), a slot's path (7, from slot 2 on), nowhere (400)."""
    V, batch, slots = 1003, 2, 6
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.randn((batch * slots, V), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dt)
    s = _ruled(V, batch, slots, {31: value, 20: value, 7: value, 400: value, 30: 1.5, 21: -1.5}, *rules)
    out = _run_logits(dtype, V, batch, slots, s, x)
    assert torch.all(out[:, [31, 20, 7, 400]] == value)
    check_logits(out, x.double().cpu().numpy(), s, dt, V, slots)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_process_logits_frequency_beyond_the_types_range(dtype):
    """f n that leaves fp32 is an infinity of its sign, not a NaN: 3 occurrences in the output, 2 on the path to slot 3."""
    V, slots = 1003, 6
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.randn((slots, V), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dt)
    for sign in (1.0, -1.0):
        s = _ruled(V, 1, slots, None, 1.2, sign * 3e38, 0.0)
        s["tok"][0, 3] = s["tok"][0, 2]
        out = _run_logits(dtype, V, 1, slots, s, x).float()
        assert torch.all(out[:, 31] == -sign * math.inf)
        assert torch.all(out[3:, 7] == -sign * math.inf) and torch.all(out[2, 7].abs() < math.inf)
        assert torch.all((out[:, 30] + sign * 3e38).abs() < 2e36)


def test_process_logits_keeps_every_bit_of_fp32():
    """What a rule takes off is whole: a logit of 0 under a repetition penalty alone stays 0, and one of 0 under a bias
    alone becomes the bias, for tokens of the output, the prompt, a path and none."""
    V, slots = 1003, 6
    x = torch.zeros((slots, V), device="cuda")
    out = _run_logits("f32", V, 1, slots, _ruled(V, 1, slots, None, 1.3, 0.0, 0.0), x)
    assert torch.all(out == 0)
    odd = {t: float(np.float32(1 + k * 2.0 ** -23)) for k, t in zip((1, 3, 5, 7), (31, 20, 7, 400))}
    for r in (1.3, 1.0):
        out = _run_logits("f32", V, 1, slots, _ruled(V, 1, slots, odd, r, 0.0, 0.0), x)
        for t, v in odd.items():
            assert torch.all(out[:, t].double() == v), (r, t)


@pytest.mark.parametrize("r", [1.3, 1.1, 0.7, 3.0, 1e-39, 3e38])
def test_process_logits_quotient_is_rounded_once(r):
    """x / r and x r in fp32, each the nearest number to the exact one, where no other rule is on; also for an r whose
    reciprocal fp32 cannot hold."""
    V, slots = 50021, 4
    rng = np.random.default_rng(7)
    x = (rng.standard_normal((slots, V)) * 10.0).astype(np.float32)
    x[:, ::5] = 0.0
    x[:, 1::5] *= np.float32(1e-30)
    hist = rng.permutation(V).astype(np.int32)[None, :30000]
    s = dict(tok=None, mask=None, hist=hist, hist_len=np.array([30000], np.int32), prompt_len=np.array([9000], np.int32),
             penalty=np.array([[r, 0.0, 0.0]], np.float32), bias_tok=None, bias_val=None, grammar=None, gram_row=None)
    out = _run_logits("f32", V, 1, slots, s, cuda(x)).cpu().numpy()
    q = np.float32(r)
    with np.errstate(over="ignore"):
        want = np.where(np.isin(np.arange(V), hist[0]), np.where(x > 0, x / q, x * q), x)
    assert want.dtype == np.float32 and np.array_equal(out, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_process_logits_between_columns_of_one_buffer(dtype):
    """Input and output rows that are column ranges of one buffer do not meet, whichever comes first; ranges that do are
    refused."""
    V, batch, slots, gap = 1003, 2, 5, 13
    x, out, s, dt = logits_inputs(dtype, batch, slots, V, 60, 9, 3, 0, 0)
    eng = g.Graft(g.graft_default_config(V, batch, g.GRAFT_MODE_STATIC, g.GRAFT_F32 if dtype == "f32" else g.GRAFT_BF16))
    for src, dst in ((0, V + gap), (V + gap, 0), (0, V), (V, 0)):
        wide = torch.full((batch * slots, 2 * V + gap), 9.0, device="cuda", dtype=dt)
        wide[:, src:src + V] = x
        call_logits(eng, batch, slots, wide[:, src:src + V], wide[:, dst:dst + V], s)
        assert eng.sync() == 0
        check_logits(wide[:, dst:dst + V], x.double().cpu().numpy(), s, dt, V, slots)
        assert torch.equal(wide[:, src:src + V], x)
    for src, dst in ((0, V - 1), (V - 1, 0), (1, 2), (V + gap, gap + 1)):
        with pytest.raises(g.GraftError) as e:
            call_logits(eng, batch, slots, wide[:, src:src + V], wide[:, dst:dst + V], s)
        assert e.value.code == gb.GRAFT_EINVAL
    assert eng.sync() == 0


def test_process_logits_bad_data_is_flagged():
    x, out, s, dt = logits_inputs("bf16", 2, 3, 500, 20, 4, 2, 0, 0)
    eng = g.Graft(g.graft_default_config(500, 2, g.GRAFT_MODE_STATIC, g.GRAFT_BF16))

    def flags(**change):
        t = {k: None if v is None else v.copy() for k, v in s.items()}
        for k, (at, value) in change.items():
            t[k][at] = value
        call_logits(eng, 2, 3, x, out, t)
        return eng.sync(raise_on_error=False)

    s["hist_len"][:] = 20
    assert flags() == 0
    assert flags(hist=((1, 3), 500)) == gb.GRAFT_ERR_TOKEN
    assert flags(hist=((0, 19), -1)) == gb.GRAFT_ERR_TOKEN
    assert flags(bias_tok=((0, 2), 501)) == gb.GRAFT_ERR_TOKEN
    assert flags(tok=((1, 0), 500)) == gb.GRAFT_ERR_TOKEN
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert flags(penalty=((1, 0), bad)) == gb.GRAFT_ERR_RULE
    assert flags(penalty=((0, 2), float("nan"))) == gb.GRAFT_ERR_RULE
    assert flags(gram_row=((0, 1), 2)) == gb.GRAFT_ERR_RULE
    assert flags(hist_len=(1, 21)) == gb.GRAFT_ERR_RULE
    with pytest.raises(g.GraftError, match="rule 1"):
        s["gram_row"][0, 0] = -2
        call_logits(eng, 2, 3, x, out, s)
        eng.sync()


def test_process_logits_then_verify():
    """A grammar that allows one successor a slot decides the verification, whatever the logits say."""
    V, B, S = 1000, 2, 61
    eng = g.Graft(g.graft_default_config(V, B, g.GRAFT_MODE_CHECKPOINT, g.GRAFT_BF16))
    tok = torch.arange(B * S, device="cuda", dtype=torch.int32).view(B, S)
    parent = torch.arange(-1, S - 1, device="cuda", dtype=torch.int32).repeat(B, 1).to(torch.int8)
    pos = torch.arange(S, device="cuda", dtype=torch.int32).repeat(B, 1)
    mask = torch.tensor([(1 << (i + 1)) - 1 for i in range(S)], device="cuda").repeat(B, 1)
    logits = torch.randn((B * S, V), device="cuda").bfloat16()
    logits[::3] = float("nan")
    table = np.zeros((B * S, (V + 31) // 32), np.uint32)
    for row in range(B * S):
        v = (row + 1) % V if row % S < 20 else 999       # the chain's next token for the first 20 slots
        table[row, v >> 5] = np.uint32(1 << (v & 31))
    logits[torch.arange(B * S), torch.tensor([(r + 1) % V if r % S < 20 else 999 for r in range(B * S)])] = -50.0
    rows = torch.arange(B * S, device="cuda", dtype=torch.int32).view(B, S)
    out = torch.empty_like(logits)
    eng.process_logits(B, S, logits, out, tree_tok=tok, tree_mask=mask, grammar=cuda(table.view(np.int32)),
                       grammar_row=rows)
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    emitted = torch.empty((B, S), dtype=torch.int32, device="cuda")
    eng.verify_update(B, tok, parent, pos, mask, out, acc, emitted)
    assert eng.sync() == 0
    assert acc.tolist() == [20, 20]
    assert emitted[0, :21].tolist() == list(range(1, 21)) + [999]


def test_calls_are_the_same_without_the_extension():
    """The binding's own form of a call (when the extension is not built, or an argument is not its usual kind) does what
    the extension's does; a closed handle refuses."""
    rng, gen = np.random.default_rng(8), torch.Generator(device="cuda").manual_seed(8)
    pre, table, pages = tables(rng, 2, 120, 40, 16)
    q, k, v = (torch.randn((10, w * 64), generator=gen, device="cuda", dtype=torch.bfloat16) for w in (4, 2, 2))
    rope, mask = torch.rand((300, 64), generator=gen, device="cuda"), torch.full((2, 5), 31, device="cuda")
    table, pre, ctx = cuda(table), cuda(pre), cuda(np.array([100, 3], np.int32))
    kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 16, pages, 2, 5))
    x = torch.randn((10, 700), generator=gen, device="cuda").bfloat16()
    eng = g.Graft(g.graft_default_config(700, 2, g.GRAFT_MODE_STATIC, g.GRAFT_BF16))
    hist = cuda(rng.integers(0, 700, (2, 9)).astype(np.int32))
    results = []
    for fast in (True, False):
        if not fast:
            kv._append = kv._attend = eng._fast = None
        kc, vc = (make_cache(torch.Generator(device="cuda").manual_seed(1), pages, 2, 16, 64, torch.bfloat16, "head") for _ in range(2))
        qo, out, lse, y = torch.empty_like(q), torch.empty_like(q), torch.empty((10, 4), device="cuda"), torch.empty_like(x)
        kv.append(2, 5, q, k, v, rope, table, ctx, kc, vc, qo, prefix_len=40)
        kv.attend(2, 5, qo, kc, vc, table, ctx, 100, out, prefix_pages=pre, prefix_len=40, tree_mask=mask, lse=lse)
        kv.attend(2, 5, qo, kc, vc, table, ctx, 100, out, prefix_pages=pre, prefix_len=40, tree_mask=mask.view(torch.uint64), lse=lse)
        eng.process_logits(2, 5, x, y, hist=hist, hist_len=cuda(np.array([9, 4], np.int32)),
                           penalty=torch.full((2, 3), 1.5, device="cuda"))
        results.append((kc, vc, qo, out, lse, y))
        assert kv.sync() == 0 and eng.sync() == 0
    assert all(torch.equal(a, b) for a, b in zip(*results))
    for h, f in ((kv, lambda: kv.attend(2, 5, q, kc, vc, table, ctx, 100, out)), (eng, lambda: eng.process_logits(2, 5, x, y))):
        h.close()
        with pytest.raises(g.GraftError) as e:
            f()
        assert e.value.code == gb.GRAFT_EINVAL


def test_attend_refuses_more_keys_than_it_counts():
    """Prefix, context and tree together stay below 2^31 keys; pages may repeat, so the tables alone would allow more."""
    kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 128, 4, 1, 4))
    k = torch.zeros((4, 2, 128, 64), device="cuda", dtype=torch.bfloat16)
    q = torch.zeros((4, 256), device="cuda", dtype=torch.bfloat16)
    table = torch.zeros((1, 1 << 24), device="cuda", dtype=torch.int32)
    ctx = torch.zeros(1, device="cuda", dtype=torch.int32)
    most = 2 ** 31 - 257
    for prefix, max_ctx in ((0, most - 3), (most - 3, 0), (most - 103, 100), (2 ** 31 - 1, 0), (0, 2 ** 31 - 5),
                            (2 ** 31 - 1, 2 ** 31 - 5)):
        with pytest.raises(g.GraftError, match="more than") as e:
            kv.attend(1, 4, q, k, k, table, ctx, max_ctx, torch.empty_like(q), prefix_pages=table.view(-1), prefix_len=prefix)
        assert e.value.code == gb.GRAFT_EINVAL
    out, lse = torch.empty_like(q), torch.empty((4, 4), device="cuda")
    kv.attend(1, 4, q, k, k, table, ctx, most - 4, out, lse=lse)      # the bound itself: the lengths are short
    assert kv.sync() == 0
    assert torch.allclose(lse, torch.arange(1, 5, device="cuda").log()[:, None].expand(4, 4), atol=1e-5)


# ------------------------------------------------------------------------------------------------------- refusals
def test_refusals_of_live_handles():
    """Argument errors come back at once, name themselves and queue nothing."""
    bf = torch.bfloat16
    kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 16, 8, 2, 4))
    k = torch.zeros((8, 2, 16, 64), device="cuda", dtype=bf)
    q, kk = torch.zeros((8, 256), device="cuda", dtype=bf), torch.zeros((8, 128), device="cuda", dtype=bf)
    rope = torch.zeros((32, 64), device="cuda")
    table, ctx = torch.zeros((2, 2), device="cuda", dtype=torch.int32), torch.zeros(2, device="cuda", dtype=torch.int32)

    def attend(batch=2, slots=4, q=q, k=k, table=table, max_ctx=28, out=None, **kw):
        kv.attend(batch, slots, q, k, k, table, ctx, max_ctx, torch.empty_like(q) if out is None else out, **kw)

    def append(batch=2, slots=4, q=q, kk=kk, rope=rope, table=table, kc=k, q_out=None, **kw):
        kv.append(batch, slots, q, kk, kk, rope, table, ctx, kc, kc, torch.empty_like(q) if q_out is None else q_out, **kw)

    attend()
    append()
    attend(batch=0)
    append(batch=0)
    bad = [lambda: attend(batch=3), lambda: attend(slots=5), lambda: attend(max_ctx=29), lambda: attend(max_ctx=-1),
           lambda: attend(scale=0.0), lambda: attend(scale=float("nan")), lambda: attend(prefix_len=-1),
           lambda: attend(prefix_len=5), lambda: attend(q=q.half()), lambda: attend(q=q[:, :255]),
           lambda: attend(k=k[:7]), lambda: attend(table=table.long()), lambda: attend(q=q.cpu(), out=q),
           lambda: append(slots=0), lambda: append(batch=-1), lambda: append(rope=rope[:, :62]),
           lambda: append(rope=None), lambda: append(prefix_len=-1), lambda: append(kk=kk[:7]),
           lambda: append(q_out=q[:7]), lambda: append(pos=torch.zeros(7, device="cuda", dtype=torch.int32)),
           lambda: kv.append(2, 4, q, kk, kk, rope, table, ctx, k, k, None),
           lambda: append(kc=torch.zeros(k.numel() + 1, device="cuda", dtype=bf)[1:])]
    for n, f in enumerate(bad):
        with pytest.raises(g.GraftError) as e:
            f()
        assert e.value.code == gb.GRAFT_EINVAL, n
        assert n < 4 or str(e.value)
    assert kv.sync() == 0
    eng = g.Graft(g.graft_default_config(100, 2, g.GRAFT_MODE_STATIC, g.GRAFT_BF16))
    x = torch.zeros((8, 100), device="cuda", dtype=bf)
    i32 = lambda *s: torch.zeros(s, device="cuda", dtype=torch.int32)  # noqa: E731
    eng.process_logits(2, 4, x, x)
    eng.process_logits(0, 4, x, x)
    wide = torch.zeros((9, 100), device="cuda", dtype=bf)
    for f in (lambda: eng.process_logits(2, 65, x, x), lambda: eng.process_logits(2, 0, x, x),
              lambda: eng.process_logits(-1, 4, x, x), lambda: eng.process_logits(2, 4, wide[:8], wide[1:]),
              lambda: eng.process_logits(2, 4, x.float(), x), lambda: eng.process_logits(2, 4, x[:7], x),
              lambda: eng.process_logits(2, 4, x, x, tree_tok=i32(2, 4)),
              lambda: eng.process_logits(2, 4, x, x, hist=i32(2, 5)),
              lambda: eng.process_logits(2, 4, x, x, hist=i32(10), hist_len=i32(2)),
              lambda: eng.process_logits(2, 4, x, x, bias_tok=i32(2, 3)),
              lambda: eng.process_logits(2, 4, x, x, bias_tok=i32(2, 2047), bias_val=torch.zeros((2, 2047), device="cuda")),
              lambda: eng.process_logits(2, 4, x, x, grammar=i32(1, 4)),
              lambda: eng.process_logits(2, 4, x, x, grammar=i32(1, 3), grammar_row=i32(2, 4)),
              lambda: eng.process_logits(2, 4, x, x, penalty=torch.zeros((2, 2), device="cuda"))):
        with pytest.raises(g.GraftError) as e:
            f()
        assert e.value.code == gb.GRAFT_EINVAL
    assert eng.sync() == 0
