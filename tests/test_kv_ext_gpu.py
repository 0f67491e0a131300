"""The paged cache in 8 bits (append, read back, attention), positions of several axes, and capped, windowed and
distance-biased scores, against plain implementations in 64 bits.

Tolerances follow from the number formats: u = 2^-8 (bf16) or 2^-11 (f16) is the largest relative error of one rounding
to the type, e = 2^-24 that of an fp32 operation; each test adds up the roundings of its formula.
"""
import math
import time
import time

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import hybrid_draft_tree_gb300 as g  # noqa: E402
from hybrid_draft_tree_gb300 import graft as gb  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
GDT = {"bf16": g.GRAFT_BF16, "f16": g.GRAFT_F16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
E = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.cuda.set_device(0)


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# every e4m3 number from its definition, by code; NaN for 0x7F and 0xFF
NUMBERS = np.array([(-1.0 if c >> 7 else 1.0) * (((c & 7) + 8) * 2.0 ** ((c >> 3 & 15) - 10) if c >> 3 & 15 else (c & 7) * 2.0 ** -9)
                    if c & 127 != 127 else math.nan for c in range(256)])


def nearest(x):
    """The e4m3 number next to each x (ties to the even code), 448 beyond the largest; fp64 in and out."""
    grid = NUMBERS[:127]
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    up = (a - grid[lo] > grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (hi % 2 == 0))
    return np.copysign(np.where(up, grid[hi], grid[lo]), x)


def by_token(cache, layout):
    """[page, token, head, d] of a cache; 8-bit ones as bytes, which can be indexed."""
    cache = cache.view(torch.uint8) if cache.dtype == E4M3 else cache
    return cache.transpose(1, 2) if layout == "head" else cache


def numbers(t):
    """What a cache's elements are, in 64 bits, without the scale."""
    return cuda(NUMBERS)[t.long()] if t.dtype == torch.uint8 else t.double()


def make_cache(gen, pages, hk, page, dim, dtype, layout, eight):
    shape = (pages, hk, page, dim) if layout == "head" else (pages, page, hk, dim)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return (x.float() * 60).clamp(-448, 448).to(E4M3) if eight else x


def random_trees(rng, batch, slots, pads=True):
    depth = np.full((batch, slots), -1, np.int32)
    mask = np.zeros((batch, slots), np.uint64)
    for b in range(batch):
        valid = int(rng.integers(max(1, slots - 3), slots + 1)) if pads else slots
        depth[b, 0], mask[b, 0] = 0, 1
        for i in range(1, valid):
            p = int(rng.integers(max(0, i - 6), i))
            depth[b, i] = depth[b, p] + 1
            mask[b, i] = int(mask[b, p]) | (1 << i)
    return depth, mask


def tables(rng, batch, tokens, prefix, page):
    own, pre = -(-tokens // page), -(-prefix // page)
    total = batch * own + pre + 2
    order = rng.permutation(total)[:total - 2].astype(np.int32)
    return order[:pre], order[pre:].reshape(batch, own), total


def head_scales(rng, hk):
    return cuda((2.0 ** rng.uniform(-7, -4, hk)).astype(np.float32))


# ---------------------------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,batch,slots,hq,hk,dim,page,layout,rot,inter,shift,with_q,with_rows,eight,axes", [
    ("bf16", 1, 1, 8, 2, 128, 16, "head", 128, 0, 0, True, False, True, 0),
    ("bf16", 3, 61, 32, 8, 128, 64, "head", 128, 0, 0, True, False, True, 0),
    ("f16", 4, 17, 10, 2, 64, 8, "token", 64, 0, 0, True, True, True, 0),
    ("bf16", 2, 64, 4, 4, 128, 128, "token", 64, 1, 0, True, False, True, 0),
    ("bf16", 2, 9, 6, 2, 64, 16, "head", 48, 0, 0, True, True, True, 0),      # rot / 2 no multiple of 8 elements
    ("f16", 3, 13, 8, 2, 128, 16, "head", 128, 0, 3, True, False, True, 0),   # rows off 16-byte boundaries
    ("bf16", 2, 5, 4, 2, 64, 16, "head", 0, 0, 0, True, False, True, 0),      # nothing rotates
    ("bf16", 1, 1000, 4, 2, 128, 16, "head", 128, 0, 0, True, False, True, 0),
    ("bf16", 3, 61, 32, 8, 128, 64, "head", 128, 0, 0, True, False, False, "16,24,24"),
    ("f16", 2, 17, 4, 2, 64, 16, "token", 64, 0, 0, True, True, False, "8,12,12"),   # pieces whose pairs differ
    ("bf16", 2, 17, 4, 2, 128, 16, "head", 128, 0, 0, True, True, True, "cycle"),    # neighbouring pairs on other axes
    ("bf16", 2, 9, 4, 2, 128, 16, "head", 64, 1, 0, False, True, True, "cycle"),
    ("f16", 2, 9, 4, 2, 64, 8, "head", 48, 0, 1, True, False, True, "cycle"),        # by elements
    ("bf16", 2, 9, 4, 2, 64, 8, "head", 64, 0, 0, True, False, False, "one"),        # one axis: positions as they are
    ("bf16", 1, 700, 4, 2, 128, 16, "token", 128, 0, 0, True, False, True, "eight"),
])
def test_append(dtype, batch, slots, hq, hk, dim, page, layout, rot, inter, shift, with_q, with_rows, eight, axes):
    rng = np.random.default_rng(slots * 7 + dim + rot + eight)
    gen = torch.Generator(device="cuda").manual_seed(slots)
    dt, half = DT[dtype], rot // 2
    ctx = rng.integers(0, 3 * page, batch).astype(np.int32)
    ctx[0] = 0
    prefix = int(rng.integers(0, 50))
    _, table, pages = tables(rng, batch, int(ctx.max()) + slots, 0, page)
    widths = [hq * dim, hk * dim, hk * dim]
    qkv = torch.randn((batch * slots, sum(widths) + shift), generator=gen, device="cuda", dtype=dt)[:, shift:]
    q, k, v = qkv.split(widths, 1)
    caches = [make_cache(gen, pages, hk, page, dim, dt, layout, eight) for _ in range(2)]
    before = [numbers(by_token(c, layout)).cpu().numpy() for c in caches]
    if slots <= 64:
        depth, _ = random_trees(rng, batch, slots)
        pos = cuda(depth)
    else:
        depth, pos = np.tile(np.arange(slots, dtype=np.int32), (batch, 1)), None
    rows = rng.integers(-1, slots, (batch, slots)) if with_rows else np.tile(np.arange(slots), (batch, 1))
    length = prefix + int(ctx.max()) + slots
    angle = np.arange(length)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    rope = cuda(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)) if rot else None
    kv = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, min(slots, 64), GDT[dtype], layout=layout,
                                             rot_dim=rot, rot_interleaved=inter, cache="e4m3" if eight else None))
    # the position of each pair: [batch, slots, pairs]
    place = np.repeat((prefix + ctx[:, None] + np.maximum(depth, 0))[..., None], half, 2)
    positions = None
    if axes:
        pair_axis = {"cycle": np.arange(half) % 3, "one": np.zeros(half, int), "eight": np.arange(half) // 8 % 8}.get(axes)
        if pair_axis is None:
            pair_axis = np.repeat(np.arange(3), [int(x) for x in axes.split(",")])
        given = rng.integers(0, length, (pair_axis.max() + 1, batch, slots)).astype(np.int32)
        kv.set_axes(pair_axis.tolist())
        positions, place = cuda(given), given[pair_axis].transpose(1, 2, 0)
    scales = {"k_scale": head_scales(rng, hk), "v_scale": head_scales(rng, hk)} if eight else {}
    q_out = torch.full((batch * slots, hq * dim + shift), 7.0, device="cuda", dtype=dt)[:, shift:] if with_q else None
    kv.append(batch, slots, q if with_q else None, k, v, rope, cuda(table), cuda(ctx), *caches, q_out, prefix_len=prefix,
              pos=pos, rows=cuda(rows.astype(np.int32)) if with_rows else None, positions=positions, **scales)
    assert kv.sync() == 0 and kv.last_launch_count() == 1
    cs = rope.double().cpu().numpy() if rot else np.zeros((length, 0))
    first = slice(0, rot, 2) if inter else slice(0, half)
    second = slice(1, rot, 2) if inter else slice(half, rot)

    def turned(x, b, i):
        """A row's heads rotated, and the sizes that bound the fp32 rotation's error: 4 e of |a| + |b|."""
        x = x[b * slots + i].double().cpu().numpy().reshape(-1, dim)
        c, s = cs[place[b, i], np.arange(half)], cs[place[b, i], np.arange(half) + half]
        y, size = x.copy(), np.zeros_like(x)
        y[:, first], y[:, second] = x[:, first] * c - x[:, second] * s, x[:, second] * c + x[:, first] * s
        size[:, first] = size[:, second] = np.abs(x[:, first]) + np.abs(x[:, second])
        return y, size

    got = [numbers(by_token(c, layout)).cpu().numpy() for c in caches]
    written = np.zeros(got[0].shape[:2], bool)
    for b in range(batch):
        for i in range(slots):
            r = rows[b, i]
            if r < 0 or depth[b, r] < 0:
                continue
            at = ctx[b] + i
            here = (table[b, at // page], at % page)
            written[here] = True
            y, size = turned(k, b, r)
            x = v[b * slots + r].double().cpu().numpy().reshape(-1, dim)
            if eight:
                # the quotient's fp32 rounding beside the rotation's error, then the nearest number, which grows with its
                # argument
                for z, off, name, at in ((y, 4 * E * size, "k_scale", 0), (x, 0 * x, "v_scale", 1)):
                    s = scales[name].double().cpu().numpy()[:, None]
                    low, high = (z - off) / s, (z + off) / s
                    assert np.all(got[at][here] >= nearest(low - E * np.abs(low)))
                    assert np.all(got[at][here] <= nearest(high + E * np.abs(high)))
            else:
                assert np.all(np.abs(got[0][here] - y) <= U[dt] * np.abs(y) + 4 * E * size + TINY[dt])
                assert np.array_equal(got[1][here], x)
    for old, new in zip(before, got):
        assert np.array_equal(old[~written], new[~written])
    if with_q:
        got_q = q_out.double().cpu().numpy().reshape(batch, slots, hq, dim)
        for b in range(batch):
            for i in range(slots):
                if depth[b, i] < 0:
                    assert np.all(got_q[b, i] == 7.0)
                else:
                    y, size = turned(q, b, i)
                    assert np.all(np.abs(got_q[b, i] - y) <= U[dt] * np.abs(y) + 4 * E * size + TINY[dt]), (b, i)


@pytest.mark.parametrize("rot,shift", [(0, 0), (0, 1), (64, 0)])
def test_append_eight_bits_of_every_kind_of_number(rot, shift):
    """Every e4m3 number, the middles between neighbours (ties to the even code), what is beyond 448, infinities, NaN,
    zeros of both signs, subnormal numbers: with a scale of 1 and of a power of two the codes are those of the definition."""
    mid = (NUMBERS[:126] + NUMBERS[1:127]) / 2
    x = np.concatenate([NUMBERS[:127], mid, [449, 463.99, 464, 1e4, 6e4, np.inf, np.nan, 2.0 ** -10, 2.0 ** -11, 1.0000001 * 2.0 ** -10]])
    x = np.concatenate([x, -x, np.zeros(-2 * len(x) % 64)])
    for dt in (torch.bfloat16, torch.float16):
        rows = cuda(x).to(dt).view(-1, 64)
        n = rows.shape[0]
        wide = torch.zeros((n, 64 + shift), device="cuda", dtype=dt)
        wide[:, shift:] = rows
        rope = torch.zeros((200, rot), device="cuda")
        rope[:, :rot // 2] = 1.0
        pages = -(-n // 8)
        kv = g.GraftKV(g.graft_kv_default_config(1, 1, 64, 8, pages, 1, 1, g.GRAFT_F16 if dt == torch.float16 else g.GRAFT_BF16,
                                                 cache="e4m3", rot_dim=rot))
        table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
        for scale in (None, 1.0, 0.25, 8.0):
            caches = [torch.zeros((pages, 1, 8, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
            given = None if scale is None else torch.tensor([scale], device="cuda")
            kv.append(1, n, None, wide[:, shift:], wide[:, shift:], rope if rot else None, table,
                      torch.zeros(1, dtype=torch.int32, device="cuda"), *caches, None, k_scale=given, v_scale=given)
            assert kv.sync() == 0
            want = rows.double().cpu().numpy() / (scale or 1.0)
            want = np.where(np.isnan(want), np.nan, nearest(want))
            for c in caches[1:] if rot else caches:
                codes = c.view(-1, 64)[:n].cpu().numpy()
                assert np.array_equal(NUMBERS[codes], want, equal_nan=True)
                assert np.array_equal(codes[~np.isnan(want)] >> 7, np.signbit(want[~np.isnan(want)]))
            if rot:      # turned by nothing: x + 0 y, which is NaN where the partner is not finite
                fine = np.isfinite(rows.double().cpu().numpy())
                fine &= np.roll(fine, 32, 1)
                assert np.array_equal(NUMBERS[caches[0].view(-1, 64)[:n].cpu().numpy()][fine], want[fine])


def test_append_ext_bad_data_is_flagged_and_skipped():
    hk, dim, page = 2, 64, 8
    k = torch.ones((4 * 3, hk * dim), device="cuda", dtype=torch.bfloat16)
    rope = torch.zeros((16, dim), device="cuda")
    rope[:, :dim // 2] = 1.0
    table = cuda(np.array([[0, 1], [2, 99], [3, -1], [4, 5]], np.int32))
    kv = g.GraftKV(g.graft_kv_default_config(hk, hk, dim, page, 6, 4, 3, cache="e4m3"))
    kv.set_axes([0] * 20 + [1] * 12)
    fine = np.zeros((2, 4, 3), np.int32)

    def one(ctx, positions=fine, k_scale=None, v_scale=None):
        kc, vc = (torch.zeros((6, hk, page, dim), device="cuda", dtype=E4M3) for _ in range(2))
        kv.append(4, 3, None, k, k, rope, table, cuda(np.array(ctx, np.int32)), kc, vc, None, positions=cuda(positions),
                  k_scale=k_scale, v_scale=v_scale)
        flags = kv.sync(raise_on_error=False)
        return flags, (kc.float()[:, 0, :, 0] == 1).sum(1).tolist(), vc.float()

    assert one([0, 0, 0, 0])[:2] == (0, [3, 0, 3, 3, 3, 0])
    assert one([0, 6, 6, 0])[:2] == (gb.GRAFT_ERR_RANGE, [3, 0, 2, 2, 3, 0])      # pages 99 and -1
    assert one([0, 0, 0, 15])[:2] == (gb.GRAFT_ERR_RANGE, [3, 0, 3, 3, 0, 1])     # beyond two pages
    assert one([0, 0, 0, -1])[:2] == (gb.GRAFT_ERR_RANGE, [3, 0, 3, 3, 0, 0])
    far = fine.copy()
    far[1, 0, 1], far[0, 2, 2], far[0, 3, 0] = 16, -1, 15
    assert one([0, 0, 0, 0], far)[:2] == (gb.GRAFT_ERR_RANGE, [2, 0, 3, 2, 3, 0])
    for bad in (0.0, -1.0, math.nan, math.inf):
        flags, counts, vc = one([0, 0, 0, 0], v_scale=torch.tensor([0.5, bad], device="cuda"))
        assert flags == gb.GRAFT_ERR_RULE and counts == [3, 0, 3, 3, 3, 0]
        assert torch.all(vc[0, 0, :3] == 2) and torch.all(vc[0, 1, :3] == 1)


# ------------------------------------------------------------------------------------------------------------ read
@pytest.mark.parametrize("dtype,batch,slots,hk,dim,page,layout,shift,eight", [
    ("bf16", 1, 1, 1, 64, 8, "head", 0, True),
    ("bf16", 3, 61, 8, 128, 64, "head", 0, True),
    ("f16", 5, 130, 2, 64, 16, "token", 0, True),
    ("bf16", 2, 33, 3, 128, 8, "token", 3, True),
    ("f16", 2, 33, 2, 128, 128, "head", 8, True),
    ("bf16", 3, 40, 2, 128, 16, "head", 0, False),
    ("f16", 3, 40, 5, 64, 32, "token", 1, False),
])
def test_read(dtype, batch, slots, hk, dim, page, layout, shift, eight):
    rng, gen = np.random.default_rng(slots), torch.Generator(device="cuda").manual_seed(slots)
    dt = DT[dtype]
    first = rng.integers(0, 3 * page, batch).astype(np.int32)
    count = rng.integers(0, slots + 1, batch).astype(np.int32)
    count[0], count[-1] = slots, count[-1] if batch > 1 else slots
    _, table, pages = tables(rng, batch, int(first.max()) + slots, 0, page)
    caches = [make_cache(gen, pages, hk, page, dim, dt, layout, eight) for _ in range(2)]
    if not eight:
        caches[0][0] = math.nan                       # a copy keeps what it copies
    scales = {"k_scale": head_scales(rng, hk), "v_scale": head_scales(rng, hk)} if eight else {}
    outs = [torch.full((batch * slots, hk * dim + shift), 7.0, device="cuda", dtype=dt)[:, shift:] for _ in range(2)]
    kv = g.GraftKV(g.graft_kv_default_config(hk, hk, dim, page, pages, batch, 1, GDT[dtype], layout=layout,
                                             cache="e4m3" if eight else None))
    kv.read(batch, slots, *caches, cuda(table), cuda(first), cuda(count), *outs, **scales)
    assert kv.sync() == 0 and kv.last_launch_count() == 1
    for cache, out, name in zip(caches, outs, ("k_scale", "v_scale")):
        held = by_token(cache, layout)
        got = out.view(batch, slots, hk, dim) if not shift else out.unflatten(0, (batch, slots)).unflatten(2, (hk, dim))
        for b in range(batch):
            n = int(count[b])
            at = int(first[b]) + np.arange(n)
            x = held[cuda(table[b, at // page]).long(), cuda(at % page)]
            if eight:
                # a product in fp32, then one rounding to the type
                want = numbers(x) * scales[name].double()[:, None]
                assert torch.all((got[b, :n].double() - want).abs() <= (U[dt] + 2 * E) * want.abs() + TINY[dt])
            else:
                assert torch.equal(got[b, :n].contiguous().view(torch.int16), x.contiguous().view(torch.int16))
            assert torch.all(got[b, n:] == 7.0)


def test_read_keeps_nan_codes_and_powers_of_two_exactly():
    """All 256 codes under scales that are powers of two: no rounding at all."""
    cache = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 1, 4, 64).repeat(1, 1, 2, 1)
    kv = g.GraftKV(g.graft_kv_default_config(1, 1, 64, 8, 1, 1, 1, cache="e4m3"))
    table, zero, n = (cuda(np.array([x], np.int32)) for x in (0, 0, 4))
    for scale in (1.0, 2.0 ** -9, 2.0 ** 30):
        outs = [torch.empty((4, 64), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        s = torch.tensor([scale], device="cuda")
        kv.read(1, 4, cache, cache, table.view(1, 1), zero, n, *outs, k_scale=s, v_scale=s)
        assert kv.sync() == 0
        for o in outs:
            assert np.array_equal(o.double().cpu().numpy().reshape(-1), NUMBERS * scale, equal_nan=True)


def test_read_bad_data_is_flagged_and_skipped():
    cache = torch.ones((6, 2, 8, 64), device="cuda").to(E4M3)
    table = cuda(np.array([[0, 1], [2, 99], [3, -1], [4, 5]], np.int32))
    kv = g.GraftKV(g.graft_kv_default_config(2, 2, 64, 8, 6, 4, 1, cache="e4m3"))

    def one(first, count, **scales):
        outs = [torch.zeros((12, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        kv.read(4, 3, cache, cache, table, cuda(np.array(first, np.int32)), cuda(np.array(count, np.int32)), *outs, **scales)
        flags = kv.sync(raise_on_error=False)
        assert torch.equal(outs[0], outs[1])
        return flags, (outs[0][:, 70] == 1).view(4, 3).sum(1).tolist()

    assert one([0, 0, 0, 0], [3, 2, 1, 0]) == (0, [3, 2, 1, 0])
    assert one([0, 6, 7, 0], [3, 3, 3, 3]) == (gb.GRAFT_ERR_RANGE, [3, 2, 1, 3])
    assert one([0, 0, 0, 15], [3, 3, 3, 3]) == (gb.GRAFT_ERR_RANGE, [3, 3, 3, 1])
    assert one([0, -1, 0, 0], [3, 3, 3, 3]) == (gb.GRAFT_ERR_RANGE, [3, 0, 3, 3])
    assert one([0, 0, 0, 0], [3, -1, 4, 3]) == (gb.GRAFT_ERR_RANGE, [3, 0, 3, 3])
    assert one([0, 0, 0, 2 ** 31 - 1], [3, 3, 3, 3]) == (gb.GRAFT_ERR_RANGE, [3, 3, 3, 0])
    bad = torch.tensor([1.0, math.nan], device="cuda")
    assert one([0, 0, 0, 0], [3, 2, 1, 0], k_scale=bad, v_scale=bad) == (gb.GRAFT_ERR_RULE, [3, 2, 1, 0])


# ---------------------------------------------------------------------------------------------------------- attend
def attend_reference(q, kt, vt, ks, vs, pre, table, prefix, ctx, mask, page, hq, hk, scale, cap, window, slopes):
    """out and lse in 64 bits, and what bounds them: the weighted sum of |v|, the largest sum |q k| of a row, and the largest
    bias of a key whose weight counts."""
    batch, slots = mask.shape
    dim, group = kt.shape[-1], hq // hk
    out = torch.zeros((batch, slots, hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((batch, slots, hq), -math.inf, dtype=torch.float64, device="cuda")
    spread, reach, bias = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    qd = q.double().view(batch, slots, hk, group, dim)
    for b in range(batch):
        shared, own = np.arange(prefix), np.arange(ctx[b] + slots)
        before = np.stack([np.concatenate([pre[shared // page] if prefix else shared, table[b, own // page]]),
                           np.concatenate([shared % page, own % page])]).astype(np.int64)
        for i in range(slots):
            path = [j for j in range(slots) if int(mask[b, i]) >> j & 1]
            if not path:
                continue
            places = np.concatenate([before[:, :prefix + ctx[b]], before[:, prefix + ctx[b] + np.array(path)]], 1)
            if window:
                places = places[:, -window:]
            at, distance = cuda(places), cuda(np.arange(places.shape[1])[::-1].astype(np.float64))
            k, v = (numbers(x[at[0], at[1]]) * y[:, None] for x, y in ((kt, ks), (vt, vs)))       # [n, hk, dim]
            s = torch.einsum("hgd,nhd->hgn", qd[b, i], k) * scale
            size = torch.einsum("hgd,nhd->hgn", qd[b, i].abs(), k.abs()).amax(-1) * scale
            if cap:
                s = cap * torch.tanh(s / cap)
            off = slopes.view(hk, group, 1) * distance
            s = s - off
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - z[..., None])
            out[b, i] = torch.einsum("hgn,nhd->hgd", w, v).reshape(hq, dim)
            spread[b, i] = torch.einsum("hgn,nhd->hgd", w, v.abs()).reshape(hq, dim)
            lse[b, i], reach[b, i] = z.reshape(hq), size.reshape(hq)
            bias[b, i] = (off.abs() * (w > 1e-13)).amax(-1).reshape(hq)
    return out, lse, spread, reach, bias


def check_attend(got, got_lse, ref, dt, keys, cap=0.0):
    out, lse, spread, reach, bias = ref
    dim = out.shape[-1]
    got = got.double().reshape(out.shape)
    # a score's fp32 sum of dim products, its scalings and the exponent's argument: (dim + 8) e of sum |q k|; the cap: the
    # exponential and the reciprocal to 2 and 1 units in the last place, the sum and the product, 16 e of it; the bias: its
    # product, its sums with score and base, 4 e; a weight is rounded to the type (u); sums over the keys and rescalings:
    # keys e; the result is rounded to the type (u)
    weight = (dim + 8) * E * (reach + 16) + 16 * E * cap + 4 * E * bias
    slack = (U[dt] + 2 * weight[..., None] + (keys + 64) * E) * spread + U[dt] * out.abs() + TINY[dt] * 2
    finite = torch.isfinite(out)
    assert torch.equal(torch.isfinite(got), finite)
    assert torch.all(((got - out).abs() <= slack)[finite])
    if got_lse is not None:
        z = got_lse.double().view(lse.shape)
        empty = lse == -math.inf
        assert torch.equal(z == -math.inf, empty)
        assert torch.all(((z - lse).abs() <= weight + (keys + 16) * E + 2 * E * lse.abs())[~empty])


def run_attend(dtype, batch, slots, prefix, ctx, hq, hk, dim, page, layout, eight, cap=0.0, window=0, alibi=0.0, causal=False,
               shift=0, scale=None, seed=0, tweak=None, max_ctx=None, q_scale=2.0, check=True):
    rng = np.random.default_rng(seed + slots * 3 + prefix)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    dt = DT[dtype]
    ctx = np.array(ctx, np.int32)
    pre, table, pages = tables(rng, batch, int(max(ctx.max(), max_ctx or 0)) + slots, prefix, page)
    caches = [make_cache(gen, pages, hk, page, dim, dt, layout, eight) for _ in range(2)]
    scales = {"k_scale": head_scales(rng, hk), "v_scale": head_scales(rng, hk)} if eight else {}
    q = (torch.randn((batch * slots, hq * dim + shift), generator=gen, device="cuda", dtype=dt) * q_scale)[:, shift:]
    slopes = cuda((alibi * 2.0 ** -rng.uniform(0, 6, hq)).astype(np.float32)) if alibi else None
    if causal:
        mask = np.array([[(1 << (i + 1)) - 1 for i in range(slots)]] * batch, np.uint64)
    else:
        _, mask = random_trees(rng, batch, slots)
    kt, vt = (by_token(c, layout) for c in caches)
    if tweak:
        tweak(rng, q, kt, vt, pre, table, ctx, mask, page)
    out = torch.full((batch * slots, hq * dim + shift), 3.0, device="cuda", dtype=dt)[:, shift:]
    lse = torch.full((batch * slots, hq), 3.0, device="cuda")
    kv = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, slots, GDT[dtype], layout=layout,
                                             cache="e4m3" if eight else None))
    kv.attend(batch, slots, q, *caches, cuda(table), cuda(ctx), int(ctx.max()) if max_ctx is None else max_ctx, out,
              prefix_pages=cuda(pre) if prefix else None, prefix_len=prefix,
              tree_mask=None if causal else cuda(mask.view(np.int64)), scale=scale, lse=lse, softcap=cap, window=window,
              slopes=slopes, **scales)
    assert kv.sync() == 0
    if check:
        one = torch.ones(hk, dtype=torch.float64, device="cuda")
        ref = attend_reference(q, kt, vt, scales["k_scale"].double() if eight else one, scales["v_scale"].double() if eight else one,
                               pre, table, prefix, ctx, mask, page, hq, hk, dim ** -0.5 if scale is None else scale, cap, window,
                               torch.zeros(hq, dtype=torch.float64, device="cuda") if slopes is None else slopes.double())
        check_attend(out, lse, ref, dt, prefix + int(ctx.max()) + slots, cap)
    return out, lse, kv


FORMS = [
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


def form_id(c):
    return f"{c[0]}-b{c[1]}-s{c[2]}-p{c[3]}-h{c[5]}x{c[6]}-d{c[7]}-g{c[8]}{c[9]}"


@pytest.mark.parametrize("case", FORMS, ids=form_id)
def test_attend_eight_bits(case):
    run_attend(*case, True)


@pytest.mark.parametrize("shape", [dict(cap=5.0), dict(window=150), dict(alibi=0.7), dict(cap=3.0, window=40, alibi=0.3)],
                         ids=lambda s: "-".join(s))
@pytest.mark.parametrize("case", FORMS, ids=form_id)
def test_attend_shaped_scores(case, shape):
    run_attend(*case, False, **shape)


@pytest.mark.parametrize("shape", [dict(cap=5.0), dict(window=150), dict(alibi=0.7), dict(cap=3.0, window=40, alibi=0.3)],
                         ids=lambda s: "-".join(s))
@pytest.mark.parametrize("case", FORMS[1::2], ids=form_id)
def test_attend_eight_bits_and_shaped_scores(case, shape):
    run_attend(*case, True, **shape)


@pytest.mark.parametrize("window", [1, 2, 3, 60, 64, 65, 127, 128, 129, 300, 384, 499, 500, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("eight", [False, True])
def test_attend_windows_of_every_kind(window, eight):
    """Windows inside the tree, that end in the context, at its first key, inside the prefix, before it; a chain of 64 slots
    and trees, contexts that end inside a block and at its end."""
    run_attend("bf16", 3, 61, 130, [240, 256, 0], 4, 2, 128, 16, "head", eight, window=window)
    run_attend("f16", 2, 64, 0, [435, 60], 4, 4, 64, 32, "token", eight, window=window, causal=True)
    run_attend("bf16", 3, 1, 500, [1, 128, 0], 8, 2, 128, 64, "head", eight, window=window)


def test_attend_a_window_of_everything_changes_nothing():
    case = ("bf16", 3, 17, 300, [700, 30, 0], 8, 2, 128, 16, "head", False)
    plain, whole = run_attend(*case), run_attend(*case, window=10 ** 6)
    assert torch.equal(plain[0], whole[0]) and torch.equal(plain[1], whole[1])


@pytest.mark.parametrize("cap,q_scale", [(0.01, 2.0), (30.0, 40.0), (50.0, 3000.0), (1e4, 2.0)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_caps_far_below_and_above_the_scores(cap, q_scale, dim):
    run_attend("bf16", 2, 5, 200, [300, 40], 8, 2, dim, 16, "head", False, cap=cap, q_scale=q_scale)
    run_attend("f16", 1, 1, 0, [1000], 4, 1, dim, 16, "head", True, cap=cap, q_scale=min(q_scale, 1000.0))


@pytest.mark.parametrize("slopes", ["steep", "rising", "zero"])
def test_attend_slopes(slopes):
    """A slope that leaves the row its own key only, negative ones (the bias grows into the past), zeros."""
    alibi = {"steep": 3e4, "rising": -0.5, "zero": 1e-30}[slopes]
    for eight in (False, True):
        run_attend("bf16", 2, 33, 140, [600, 30], 8, 4, 128, 16, "head", eight, alibi=alibi)
        run_attend("bf16", 2, 1, 140, [600, 30], 8, 4, 64, 16, "head", eight, alibi=alibi)


def test_attend_without_a_mask_or_lse_and_at_any_row_offset():
    for shift in (0, 1, 8):
        run_attend("bf16", 2, 9, 30, [33, 250], 8, 2, 128, 16, "token", True, shift=shift, causal=True)
        run_attend("f16", 2, 9, 30, [33, 250], 8, 2, 64, 16, "token", False, shift=shift, causal=True, cap=4.0, window=99)


def test_attend_ext_ctx_bound_above_every_length():
    for more in (dict(eight=True), dict(eight=False, window=333), dict(eight=True, cap=9.0, alibi=0.1)):
        run_attend("bf16", 3, 3, 0, [0, 5, 300], 8, 2, 128, 16, "head", max_ctx=9000, **more)
        run_attend("bf16", 3, 1, 500, [0, 5, 300], 8, 2, 128, 16, "head", max_ctx=9000, **more)
        run_attend("f16", 2, 61, 90, [0, 129], 8, 2, 64, 16, "token", max_ctx=5000, **more)


def test_attend_large_scores_and_a_rising_maximum():
    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        for b in range(len(ctx)):
            for at in range(int(ctx[b])):
                here = k[table[b, at // page], at % page]
                here.copy_((here.view(E4M3).float() * (0.02 + at / 900.0)).clamp(-448, 448).to(E4M3).view(torch.uint8))
    run_attend("bf16", 2, 4, 0, [1500, 900], 4, 2, 128, 64, "head", True, tweak=tweak, q_scale=8.0)
    run_attend("f16", 2, 61, 0, [1500, 900], 4, 2, 64, 16, "head", True, tweak=tweak, scale=1.0)


def test_attend_ext_masks_that_leave_nothing():
    """Pads give zeros and -inf; a mask without the slot's own bit; a window that leaves such a row its last key."""
    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        mask[0, :] = 0
        mask[1, 2] = 1 << 1
        mask[1, 3] = 0
    for more in (dict(eight=True), dict(eight=False, window=1), dict(eight=True, cap=2.0, alibi=0.5)):
        out, lse, _ = run_attend("bf16", 2, 5, 0, [40, 0], 4, 2, 128, 16, "head", tweak=tweak, **more)
        assert torch.all(out[:5] == 0) and torch.all(lse[:5] == -math.inf) and torch.all(out[8] == 0)


@pytest.mark.parametrize("eight,value", [(False, math.nan), (False, math.inf), (False, -math.inf), (True, math.nan)])
@pytest.mark.parametrize("window", [0, 1, 30, 90, 200])
@pytest.mark.parametrize("dims", [(2, 9, 37, [130, 61]), (3, 1, 200, [20, 0, 100]), (1, 61, 0, [1000]), (1, 64, 190, [70])])
def test_attend_what_is_not_seen_has_no_effect(value, eight, window, dims):
    """Everything that no slot of a request sees is NaN or infinite (8-bit caches: NaN): the rest of its pages, keys before
    every window, the pads' slots, pages of nobody.  Pads' queries are too."""
    unseen_has_no_effect(value, eight, dims, window=window)


@pytest.mark.parametrize("eight,value", [(False, math.nan), (False, math.inf), (True, math.nan)])
@pytest.mark.parametrize("shape", [dict(cap=0.5), dict(cap=300.0), dict(alibi=0.5), dict(cap=0.5, window=90, alibi=0.1)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
@pytest.mark.parametrize("dims", [(2, 9, 37, [130, 61]), (3, 1, 200, [20, 0, 100]), (1, 61, 0, [1000])])
def test_attend_what_is_not_seen_has_no_effect_on_shaped_scores(eight, value, shape, dims):
    unseen_has_no_effect(value, eight, dims, **shape)


def unseen_has_no_effect(value, eight, dims, window=0, **shape):
    batch, slots, prefix, ctx = dims

    def tweak(rng, q, k, v, pre, table, ctx, mask, page):
        keep = torch.zeros(k.shape[:2], dtype=torch.bool)
        for b in range(batch):
            for i in range(slots):
                path = [j for j in range(slots) if int(mask[b, i]) >> j & 1]
                if not path:
                    q[b * slots + i] = value
                    continue
                places = [(pre[p // page], p % page) for p in range(prefix)]
                places += [(table[b, p // page], p % page) for p in [*range(ctx[b]), *(int(ctx[b]) + j for j in path)]]
                for p, o in places[-window if window else 0:]:
                    keep[p, o] = True
        for x in (k, v):
            x[~keep.cuda()] = 0x7F if eight else value
    run_attend("bf16", batch, slots, prefix, ctx, 8, 2, 128, 16, "head", eight, window=window, tweak=tweak, **shape)
    run_attend("f16", batch, slots, prefix, ctx, 8, 2, 64, 16, "token", eight, window=window, tweak=tweak, **shape)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("slots", [3, 40])
@pytest.mark.parametrize("shape", [dict(), dict(cap=0.5), dict(cap=300.0), dict(alibi=0.2), dict(cap=0.5, alibi=0.2, window=60)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_attend_keys_that_are_no_numbers_reach_only_those_that_see_them(eight, slots, shape):
    """A slot's key that is a NaN spoils the rows that see it and leaves every bit of the others."""
    seen = {}

    def spoil(rng, q, k, v, pre, table, ctx, mask, page):
        j = slots // 2
        at = int(ctx[0]) + j
        k[table[0, at // page], at % page, 0, 7] = 0x7F if eight else math.nan
        seen["rows"] = torch.tensor([int(m) >> j & 1 for m in mask[0]], dtype=torch.bool, device="cuda")
    args = ("bf16", 1, slots, 0, [150], 8, 2, 128, 16, "head", eight)
    clean = run_attend(*args, **shape)[0].view(slots, 8, 128)
    out = run_attend(*args, **shape, tweak=spoil, check=False)[0].view(slots, 8, 128)
    assert torch.equal(out[:, 4:], clean[:, 4:]) and torch.equal(out[~seen["rows"]], clean[~seen["rows"]])
    assert seen["rows"].any() and not torch.isfinite(out[seen["rows"]][:, :4]).any()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("window", [0, 20, 100])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
def test_attend_non_finite_values_reach_only_those_that_see_them(eight, window, dtype, dim):
    """Values of slots, and of keys that some rows' windows hold and others' do not, that are not finite."""
    batch, slots, prefix, ctx, page = 2, 40, 50, [100, 47], 16

    def spoil(rng, q, k, v, pre, table, ctx, mask, page):
        spots = [(b, prefix + int(ctx[b]) + j) for b, j in ((0, 5), (0, 17), (1, 30), (1, 11))]
        if window:                      # the edge of the windows, from the root's to the deepest slot's
            spots += [(0, prefix + int(ctx[0]) - window + d) for d in (2, 4, 7)]
            spots += [(1, prefix + int(ctx[1]) - window + d) for d in (1, 3)]
        for b, at in spots:
            where = (pre[at // page], at % page) if at < prefix else (table[b, (at - prefix) // page], (at - prefix) % page)
            v[where[0], where[1], 0, 3] = 0x7F if eight else math.inf
            v[where[0], where[1], 0, dim - 1] = 0xFF if eight else math.nan
    clean = run_attend(dtype, batch, slots, prefix, ctx, 8, 2, dim, page, "head", eight, window=window)
    out = run_attend(dtype, batch, slots, prefix, ctx, 8, 2, dim, page, "head", eight, window=window, tweak=spoil)
    a, b = (x[0].view(batch * slots, 8, dim) for x in (clean, out))
    assert torch.equal(a[:, 4:], b[:, 4:])                                # heads of kv head 1
    rest = [d for d in range(dim) if d not in (3, dim - 1)]
    assert torch.equal(a[:, :4, rest], b[:, :4, rest])
    assert not torch.isfinite(b[:, :4, 3]).all() and torch.isfinite(b[:, :4, 3]).any()
    assert torch.equal(clean[1], out[1])


def test_attend_ext_bad_data_is_flagged_and_stays_in_bounds():
    rng, gen = np.random.default_rng(4), torch.Generator(device="cuda").manual_seed(4)
    _, table, pages = tables(rng, 2, 300, 0, 16)
    q = torch.randn((2, 4 * 64), generator=gen, device="cuda", dtype=torch.bfloat16)
    for eight, more in ((True, {}), (True, dict(cap=5.0, window=200)), (False, dict(alibi=1.0))):
        caches = [make_cache(gen, pages, 2, 16, 64, torch.bfloat16, "head", eight) for _ in range(2)]
        kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 16, pages, 2, 1, cache="e4m3" if eight else None))
        slopes = torch.full((4,), 0.25, device="cuda") if "alibi" in more else None
        shape = dict(softcap=more.get("cap", 0.0), window=more.get("window", 0))

        def call(tab=table, ctx=(290, 100), slopes=slopes, **scales):
            out = torch.full_like(q, 9.0)
            kv.attend(2, 1, q, *caches, cuda(tab), cuda(np.array(ctx, np.int32)), 290, out, slopes=slopes, **shape, **scales)
            return kv.sync(raise_on_error=False), out

        flags, want = call()
        assert flags == 0
        flags, out = call(ctx=(1000, 100))                                   # clamped to the bound
        assert flags == gb.GRAFT_ERR_RANGE and torch.equal(out, want)
        flags, out = call(ctx=(290, -7))
        assert flags == gb.GRAFT_ERR_RANGE and torch.equal(out[0], want[0]) and torch.isfinite(out).all()
        wrong = table.copy()
        wrong[1, 2], wrong[1, 3] = pages, -5                                 # read as zeros
        flags, out = call(wrong)
        assert flags == gb.GRAFT_ERR_RANGE and torch.equal(out[0], want[0]) and torch.isfinite(out).all()
        if eight:
            for bad in (0.0, math.nan, -2.0, math.inf):
                good = torch.tensor([1.0, 0.5], device="cuda")
                half = torch.tensor([bad, 0.5], device="cuda")
                flags, out = call(k_scale=half, v_scale=half)
                assert flags == gb.GRAFT_ERR_RULE and torch.equal(out, call(k_scale=good, v_scale=good)[1])
        if slopes is not None:
            for bad in (math.nan, math.inf):
                flags, out = call(slopes=torch.tensor([0.25, bad, 0.25, 0.25], device="cuda"))
                assert flags == gb.GRAFT_ERR_RULE
                assert torch.equal(out, call(slopes=torch.tensor([0.25, 0.0, 0.25, 0.25], device="cuda"))[1])


@pytest.mark.parametrize("slots", [1, 40])
@pytest.mark.parametrize("eight,shape", [(True, {}), (False, dict(softcap=6.0, window=500)), (True, dict(softcap=6.0, window=200))])
def test_attend_ext_repeats_bit_for_bit_and_from_a_graph_and_another_stream(slots, eight, shape):
    rng, gen = np.random.default_rng(7), torch.Generator(device="cuda").manual_seed(7)
    pre, table, pages = tables(rng, 3, 2050, 300, 16)
    caches = [make_cache(gen, pages, 2, 16, 128, torch.bfloat16, "head", eight) for _ in range(2)]
    q = torch.randn((3 * slots, 8 * 128), generator=gen, device="cuda", dtype=torch.bfloat16)
    slopes = torch.rand(8, generator=gen, device="cuda") * 0.1
    scales = {n: torch.rand(2, generator=gen, device="cuda") * 0.05 + 0.01 for n in ("k_scale", "v_scale")} if eight else {}
    kv = g.GraftKV(g.graft_kv_default_config(8, 2, 128, 16, pages, 3, slots, cache="e4m3" if eight else None))
    table, pre, ctx = cuda(table), cuda(pre), cuda(np.array([2000, 1, 700], np.int32))
    outs = [torch.zeros_like(q) for _ in range(3)]
    call = lambda o, **s: kv.attend(3, slots, q, *caches, table, ctx, 2000, o, prefix_pages=pre, prefix_len=300,  # noqa: E731
                                    slopes=slopes, **shape, **scales, **s)
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


@pytest.mark.parametrize("order", [(0, 1, 2), (1, 0, 2), (2, 0, 1), (2, 1, 0), (1, 2, 0)])
def test_eight_bit_strides_in_any_order(order):
    """Caches whose pages, heads and tokens nest in any order: append, read and attend agree with one of pages first."""
    rng, gen = np.random.default_rng(3), torch.Generator(device="cuda").manual_seed(3)
    batch, slots, hq, hk, dim, page = 2, 5, 4, 2, 64, 16
    ctx = np.array([140, 33], np.int32)
    _, table, pages = tables(rng, batch, int(ctx.max()) + slots, 0, page)
    start = [make_cache(gen, pages, hk, page, dim, torch.bfloat16, "head", True).view(torch.uint8) for _ in range(2)]
    q, k, v = (torch.randn((batch * slots, h * dim), generator=gen, device="cuda", dtype=torch.bfloat16) for h in (hq, hk, hk))
    rope = torch.rand((200, dim), generator=gen, device="cuda")
    scale = head_scales(rng, hk)
    table, at, count = cuda(table), cuda(ctx), cuda(np.array([145, 38], np.int32))

    def results(order):
        back = [order.index(a) for a in range(3)] + [3]
        caches = [x.permute(*order, 3).contiguous() for x in start]
        strides = caches[0].permute(back).stride()
        kv = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, slots, page_stride=strides[0],
                                                 head_stride=strides[1], token_stride=strides[2], cache="e4m3"))
        rot, out = torch.empty_like(q), torch.empty_like(q)
        rows = [torch.zeros((batch * 145, hk * dim), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        kv.append(batch, slots, q, k, v, rope, table, at, *caches, rot, k_scale=scale, v_scale=scale)
        kv.attend(batch, slots, rot, *caches, table, at, 140, out, k_scale=scale, v_scale=scale)
        kv.read(batch, 145, *caches, table, torch.zeros_like(at), count, *rows, k_scale=scale, v_scale=scale)
        assert kv.sync() == 0
        return [*(c.permute(back) for c in caches), rot, out, *rows]
    for got, want in zip(results(order), results((0, 1, 2))):
        assert torch.equal(got, want)


def test_eight_bit_offsets_beyond_32_bits():
    """Pages far apart in a cache of 2^32 bytes and more."""
    hk, dim, page, pages = 2, 128, 16, 5
    stride = (1 << 30) + 4096
    cache = torch.zeros((pages - 1) * stride + hk * page * dim, device="cuda", dtype=torch.uint8)
    kv = g.GraftKV(g.graft_kv_default_config(4, hk, dim, page, pages, 1, 4, page_stride=stride, cache="e4m3"))
    small = g.GraftKV(g.graft_kv_default_config(4, hk, dim, page, pages, 1, 4, cache="e4m3"))
    near = torch.zeros((pages, hk, page, dim), device="cuda", dtype=torch.uint8)
    gen = torch.Generator(device="cuda").manual_seed(9)
    k = torch.randn((36, hk * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    q = torch.randn((4, 4 * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    rope = torch.rand((64, dim), generator=gen, device="cuda")
    table = cuda(np.array([[4, 3, 1]], np.int32))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for h, c in ((kv, cache), (small, near)):
        out = torch.empty_like(q)
        rows = [torch.zeros((36, hk * dim), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        h.append(1, 36, None, k, k, rope, table, zero, c, c, None)
        h.attend(1, 4, q, c, c, table, zero + 32, 32, out, softcap=9.0, window=30)
        h.read(1, 36, c, c, table, zero, zero + 36, *rows)
        assert h.sync() == 0
        got.append([out, *rows])
    assert all(torch.equal(x, y) for x, y in zip(*got)) and got[0][1].abs().sum() > 0


def test_append_attend_and_read_agree():
    """A run of them together: what is appended in 8 bits reads back within its rounding, and the attention over it is that
    over a 16-bit cache that holds the same numbers."""
    rng, gen = np.random.default_rng(2), torch.Generator(device="cuda").manual_seed(2)
    batch, slots, ctx, hq, hk, dim, page = 2, 61, 300, 8, 2, 128, 16
    _, table, pages = tables(rng, batch, ctx + slots, 0, page)
    table = cuda(table)
    n = ctx + slots
    q = torch.randn((batch * slots, hq * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn((batch * n, hk * dim), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    zero = torch.zeros(batch, dtype=torch.int32, device="cuda")
    rope = torch.cat([torch.ones((n, dim // 2), device="cuda"), torch.zeros((n, dim // 2), device="cuda")], 1)
    scale = torch.tensor([2.0 ** -6, 2.0 ** -7], device="cuda")          # powers of two: the numbers are bf16 numbers
    s8 = dict(k_scale=scale, v_scale=scale)
    eight = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, slots, cache="e4m3"))
    caches = [torch.zeros((pages, hk, page, dim), dtype=E4M3, device="cuda") for _ in range(2)]
    eight.append(batch, n, None, k, v, rope, table, zero, *caches, None, **s8)
    rows = [torch.empty_like(k) for _ in range(2)]
    eight.read(batch, n, *caches, table, zero, zero + n, *rows, **s8)
    for x, y in zip((k, v), rows):
        # half a step of e4m3, or of its subnormal numbers; beyond 448 times the scale (3.5 for the second head, and normal
        # numbers pass it) the definition stores 448, which is |x| - 448 scale away
        x, y, s = x.float().view(-1, hk, dim), y.float().view(-1, hk, dim), scale[:, None]
        assert torch.all((x - y).abs() <= torch.maximum((x.abs() * 2 ** -4).clamp(min=2.0 ** -10 * 2.0 ** -6), x.abs() - 448 * s))
    wide = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, slots))
    held = [torch.zeros((pages, hk, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wide.append(batch, n, None, *rows, rope, table, zero, *held, None)
    _, mask = random_trees(rng, batch, slots)
    mask = cuda(mask.view(np.int64))
    outs = [torch.empty_like(q) for _ in range(2)]
    lses = [torch.empty((batch * slots, hq), device="cuda") for _ in range(2)]
    eight.attend(batch, slots, q, *caches, table, zero + ctx, ctx, outs[0], tree_mask=mask, lse=lses[0], **s8)
    wide.attend(batch, slots, q, *held, table, zero + ctx, ctx, outs[1], tree_mask=mask, lse=lses[1])
    assert eight.sync() == 0 and wide.sync() == 0
    # each within u of the weighted |v| (a weight's rounding) and u of itself (its own) of the same definition
    size = v.float().abs().max()
    assert torch.all((outs[0].float() - outs[1].float()).abs() <= 2 * 2 ** -8 * (size + outs[1].float().abs()))
    live = lses[1] > -math.inf
    assert torch.allclose(lses[0][live], lses[1][live], rtol=1e-5, atol=1e-4) and torch.equal(live, lses[0] > -math.inf)


def test_ext_calls_are_the_same_without_the_extension():
    """The binding's own form of a call gives what the extension's does."""
    rng, gen = np.random.default_rng(11), torch.Generator(device="cuda").manual_seed(11)
    _, table, pages = tables(rng, 2, 60, 0, 16)
    q, k, v = (torch.randn((10, h * 64), generator=gen, device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2))
    rope = torch.rand((64, 64), generator=gen, device="cuda")
    table, ctx, count = cuda(table), cuda(np.array([50, 3], np.int32)), cuda(np.array([5, 2], np.int32))
    scale = head_scales(rng, 2)
    positions = cuda(rng.integers(0, 64, (3, 2, 5)).astype(np.int32))
    slopes = torch.rand(4, generator=gen, device="cuda")
    kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 16, pages, 2, 5, cache="e4m3"))
    kv.set_axes([0, 1, 2, 0] * 8)
    start = [make_cache(gen, pages, 2, 16, 64, torch.bfloat16, "head", True).view(torch.uint8) for _ in range(2)]

    def results(kind):
        caches = [c.clone().view(kind) for c in start]
        rot, out, k_out, v_out = torch.empty_like(q), torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(k)
        kv.append(2, 5, q, k, v, rope, table, ctx, *caches, rot, positions=positions, k_scale=scale, v_scale=scale)
        kv.attend(2, 5, rot, *caches, table, ctx, 50, out, softcap=7.0, window=33, slopes=slopes, k_scale=scale, v_scale=scale)
        kv.read(2, 5, *caches, table, ctx, count, k_out, v_out, k_scale=scale, v_scale=scale)
        assert kv.sync() == 0
        return [*(c.view(torch.uint8) for c in caches), rot, out, k_out, v_out]
    assert kv._append_ext.module is not None, "the extension is not built"
    fast = results(E4M3)
    kv._append_ext = kv._attend_ext = kv._read = None
    for kind in (E4M3, torch.uint8):
        assert all(torch.equal(x, y) for x, y in zip(fast, results(kind)))


def test_ext_refusals_of_live_handles():
    kv = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 16, 8, 2, 4, cache="e4m3"))
    wide = g.GraftKV(g.graft_kv_default_config(4, 2, 64, 16, 8, 2, 4))
    x = torch.zeros((8, 256), device="cuda", dtype=torch.bfloat16)
    c8, c16 = torch.zeros((8, 2, 16, 64), device="cuda", dtype=E4M3), torch.zeros((8, 2, 16, 64), device="cuda", dtype=torch.bfloat16)
    table, ctx = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    rope, scale = torch.zeros((99, 64), device="cuda"), torch.ones(2, device="cuda")
    k = x[:, :128]

    def refused(match, f):
        with pytest.raises(g.GraftError, match=match) as e:
            f()
        assert e.value.code == gb.GRAFT_EINVAL
    for bad in (-1.0, math.nan, math.inf, 1e-35):
        refused("softcap", lambda: wide.attend(2, 4, x, c16, c16, table, ctx, 0, x, softcap=bad))
    refused("window", lambda: wide.attend(2, 4, x, c16, c16, table, ctx, 0, x, window=-1))
    refused("window", lambda: wide.attend(2, 4, x, c16, c16, table, ctx, 0, x, window=2 ** 31))
    refused("scales", lambda: wide.attend(2, 4, x, c16, c16, table, ctx, 0, x, k_scale=scale))
    refused("scales", lambda: wide.append(2, 4, x, k, k, rope, table, ctx, c16, c16, x, v_scale=scale))
    refused("scales", lambda: wide.read(2, 4, c16, c16, table, ctx, ctx, k, k, v_scale=scale))
    refused("dtype", lambda: kv.attend(2, 4, x, c16, c16, table, ctx, 0, x))
    refused("dtype", lambda: wide.attend(2, 4, x, c8, c8, table, ctx, 0, x, softcap=5.0))
    refused("dtype", lambda: kv.append(2, 4, x, k, k, rope, table, ctx, c8, c16, x))
    refused("k_scale", lambda: kv.append(2, 4, x, k, k, rope, table, ctx, c8, c8, x, k_scale=scale[:1]))
    refused("v_scale", lambda: kv.read(2, 4, c8, c8, table, ctx, ctx, k, k, v_scale=scale.double()))
    refused("slopes", lambda: kv.attend(2, 4, x, c8, c8, table, ctx, 0, x, slopes=scale))
    refused("positions", lambda: kv.append(2, 4, x, k, k, rope, table, ctx, c8, c8, x, positions=ctx))
    refused("positions", lambda: kv.append(2, 4, x, k, k, rope, table, ctx, c8, c8, x,
                                           positions=torch.zeros((2, 2, 4), dtype=torch.int32, device="cuda")))
    refused("pairs", lambda: kv.set_axes([0] * 31))
    refused("axis", lambda: kv.set_axes([0] * 31 + [-1]))
    refused("axes", lambda: kv.set_axes([0] * 31 + [8]))
    odd = torch.zeros(20000, device="cuda", dtype=torch.uint8)[1:]
    refused("16 bytes", lambda: kv.read(2, 4, odd, odd, table, ctx, ctx, k, k))
    refused("max_ctx", lambda: kv.attend(2, 4, x, c8, c8, table, ctx, 61, x))
    refused("batch", lambda: kv.attend(3, 1, x, c8, c8, torch.zeros((3, 4), dtype=torch.int32, device="cuda"),
                                       torch.zeros(3, dtype=torch.int32, device="cuda"), 0, x))
    with pytest.raises(g.GraftError, match="cache"):
        g.graft_kv_default_config(4, 2, 64, 16, 8, 2, 4, cache="int8")
    assert kv.sync() == 0 and wide.sync() == 0
    kv.append(0, 4, x, k, k, rope, table[:0], ctx[:0], c8, c8, x)
    kv.attend(0, 4, x, c8, c8, table[:0], ctx[:0], 0, x)
    kv.read(0, 4, c8, c8, table[:0], ctx[:0], ctx[:0], k, k)
    assert kv.sync() == 0 and kv.last_launch_count() == 0


@pytest.mark.parametrize("eight,slots,page,dim,shape", [
    (True, 1, 64, 128, {}), (True, 1, 8, 64, {}), (True, 3, 16, 128, dict(softcap=5.0, window=300)), (True, 12, 16, 128, {}),
    (True, 12, 8, 64, {}), (True, 40, 64, 128, {}), (True, 40, 16, 64, dict(window=200)), (False, 1, 16, 128, dict(window=300)),
    (False, 40, 64, 128, dict(softcap=5.0)), (False, 40, 16, 64, dict(softcap=5.0, window=99)),
])
def test_attend_ext_waits_are_bounded(eight, slots, page, dim, shape):
    """With limits of a few polls waits run out: the call ends at once, says so, and the handle works on.  With and without
    a prefix that the requests' rows are packed against."""
    rng, gen = np.random.default_rng(6), torch.Generator(device="cuda").manual_seed(6)
    pre, table, pages = tables(rng, 20, 700 + slots, 900, page)
    caches = [make_cache(gen, pages, 2, page, dim, torch.bfloat16, "head", eight) for _ in range(2)]
    kv = g.GraftKV(g.graft_kv_default_config(8, 2, dim, page, pages, 20, slots, cache="e4m3" if eight else None))
    table, pre, at = cuda(table), cuda(pre), cuda((np.arange(20) * 37 % 700).astype(np.int32))
    q = torch.randn((20 * slots, 8 * dim), generator=gen, device="cuda", dtype=torch.bfloat16) * 0.1
    for prefix in (0, 900):
        want, out = torch.zeros_like(q), torch.zeros_like(q)
        call = lambda o: kv.attend(20, slots, q, *caches, table, at, 700, o, prefix_pages=pre if prefix else None,  # noqa: E731
                                   prefix_len=prefix, **shape)
        call(want)
        assert kv.sync() == 0
        expired = 0
        for limit in [1, 2, 3] * 5:
            kv.set_wait_limit(limit)
            start = time.perf_counter()
            call(out)
            flags = kv.sync(raise_on_error=False)
            assert time.perf_counter() - start < 0.5
            assert flags in (0, gb.GRAFT_ERR_TIMEOUT)
            assert flags or torch.equal(out, want)
            expired += flags != 0
        # CTAs of few rows wait for copies alone, which may all land within one poll
        assert expired or (eight and slots * 4 <= 16)
        kv.set_wait_limit(0)
        out.zero_()
        call(out)
        assert kv.sync() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("scale", [2.0 ** -149, 1e-38, 3e-19, 2.0 ** -60, 0.0117, 1 / 3, 448.0, 2.0 ** 60, 5e19, 3e38])
def test_append_quotients_are_correctly_rounded(scale):
    """Codes are those of the correctly rounded fp32 quotient, whatever the scale: next to every middle between neighbours,
    and over magnitudes from the smallest to the largest."""
    rng = np.random.default_rng(1)
    s = np.float32(scale)
    middles = np.concatenate([(NUMBERS[:126] + NUMBERS[1:127]) / 2, [464.0, 448.0, 2.0 ** -10]])
    x = np.concatenate([middles * float(s) * (1 + k * 2.0 ** -8) for k in (-2, -1, 0, 1, 2)] +
                       [2.0 ** rng.uniform(-130, 127, 3000), float(s) * 2.0 ** rng.uniform(-14, 12, 3000)])
    x = np.clip(np.concatenate([x, -x, np.zeros(-2 * len(x) % 64)]), -3e38, 3e38)
    rows = cuda(x).to(torch.bfloat16).view(-1, 64)
    n = rows.shape[0]
    pages = -(-n // 128)
    kv = g.GraftKV(g.graft_kv_default_config(1, 1, 64, 128, pages, 1, 1, cache="e4m3", rot_dim=0))
    caches = [torch.zeros((pages, 1, 128, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    given = torch.tensor([s], device="cuda")
    kv.append(1, n, None, rows, rows, None, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1),
              torch.zeros(1, dtype=torch.int32, device="cuda"), *caches, None, k_scale=given, v_scale=given)
    assert kv.sync() == 0
    with np.errstate(over="ignore"):
        want = nearest((rows.float().cpu().numpy() / s).astype(np.float32))
    for c in caches:
        assert np.array_equal(NUMBERS[c.view(-1, 64)[:n].cpu().numpy()], want)


def test_append_quotients_over_rotated_keys():
    """fp32 values of every last bit (sums of two products) over scales that are no powers of two: the codes are those of
    the fp32 rotation and the quotient, each within half an ulp, so no further than the next fp32 number's."""
    rng, gen = np.random.default_rng(3), torch.Generator(device="cuda").manual_seed(3)
    n, hk, dim = 3000, 4, 64
    k = torch.randn((n, hk * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    rope = torch.rand((n, dim), generator=gen, device="cuda") * 2 - 1
    pages = -(-n // 128)
    kv = g.GraftKV(g.graft_kv_default_config(hk, hk, dim, 128, pages, 1, 1, cache="e4m3"))
    caches = [torch.zeros((pages, hk, 128, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = head_scales(rng, hk) * 0.77
    kv.append(1, n, None, k, k, rope, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1),
              torch.zeros(1, dtype=torch.int32, device="cuda"), *caches, None, k_scale=scale, v_scale=scale)
    assert kv.sync() == 0
    x, cs = k.double().cpu().numpy().reshape(n, hk, dim), rope.double().cpu().numpy()[:, None]
    a, b, c, s = x[..., :32], x[..., 32:], cs[..., :32], cs[..., 32:]
    z = np.concatenate([a * c - b * s, b * c + a * s], -1)
    off = 2 * E * np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)
    by = scale.double().cpu().numpy()[:, None]
    low, high = (z - off) / by, (z + off) / by
    got = NUMBERS[caches[0].cpu().numpy()].transpose(0, 2, 1, 3).reshape(-1, hk, dim)[:n]
    assert np.all(got >= nearest(low - E * np.abs(low))) and np.all(got <= nearest(high + E * np.abs(high)))
