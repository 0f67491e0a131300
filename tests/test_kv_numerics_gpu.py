"""Where attention's numbers are stretched: caps far above the scores, rows of very different scores beside each other, and a
first key that outweighs the others by far and counts for nothing.  Against the definition in 64 bits; tolerances add up the
roundings, e = 2^-24 an fp32 operation's, u = 2^-8 (bf16) or 2^-11 (f16) the type's."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import hybrid_draft_tree_gb300 as g  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
GDT = {"bf16": g.GRAFT_BF16, "f16": g.GRAFT_F16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
E = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.cuda.set_device(0)


def held(x, eight, dtype):
    """What a cache holds of x, as numbers and as it is."""
    kept = x.clamp(-448, 448).to(E4M3) if eight else x.to(DT[dtype])
    return kept.double(), kept


def attend(dtype, eight, q, k, v, prefix=0, page=32, **scores):
    """Rows q [batch, slots, hq, dim] after k, v [batch, keys, hk, dim], whose last `slots` are the rows' own, under causal
    masks; the first `prefix` keys are the first request's for all.  The result, its lse, the definition of both in 64 bits,
    the sum of weight times |v|, the largest weight times the sum of |v|, and the row's largest sum of |q k| and capped score."""
    (batch, slots, hq, dim), (keys, hk) = q.shape, k.shape[1:3]
    ctx = keys - slots - prefix
    q = q.to(DT[dtype])
    (kn, kc), (vn, vc) = held(k, eight, dtype), held(v, eight, dtype)
    pre, own = -(-prefix // page), -(-(keys - prefix) // page)
    pages = pre + batch * own

    def paged(x):
        cache = torch.zeros((pages * page, hk, dim), dtype=torch.uint8 if eight else x.dtype, device="cuda")
        x = x.view(torch.uint8) if eight else x
        cache[:prefix] = x[0, :prefix]
        for b in range(batch):
            at = (pre + b * own) * page
            cache[at:at + keys - prefix] = x[b, prefix:]
        return cache.view(pages, page, hk, dim).transpose(1, 2).contiguous()
    caches = paged(kc), paged(vc)
    if prefix:
        kn, vn = (torch.cat([x[:1, :prefix].expand(batch, -1, -1, -1), x[:, prefix:]], 1) for x in (kn, vn))
    kv = g.GraftKV(g.graft_kv_default_config(hq, hk, dim, page, pages, batch, slots, GDT[dtype], cache="e4m3" if eight else None))
    rows = q.reshape(batch * slots, hq * dim).contiguous()
    out, lse = torch.zeros_like(rows), torch.zeros((batch * slots, hq), device="cuda")
    table = torch.arange(pre, pages, dtype=torch.int32, device="cuda").view(batch, own)
    kv.attend(batch, slots, rows, *caches, table, torch.full((batch,), ctx, dtype=torch.int32, device="cuda"), ctx, out,
              prefix_pages=torch.arange(pre, dtype=torch.int32, device="cuda") if prefix else None, prefix_len=prefix, lse=lse, **scores)
    assert kv.sync() == 0
    place = torch.arange(keys, device="cuda")
    distance = (keys - slots + torch.arange(slots, device="cuda"))[:, None] - place
    want = {n: [] for n in ("out", "lse", "spread", "top", "reach", "score")}
    for b in range(batch):
        qd = q[b].double().view(slots, hk, hq // hk, dim)
        s = torch.einsum("shgd,nhd->shgn", qd, kn[b]) * dim ** -0.5
        reach = torch.einsum("shgd,nhd->shgn", qd.abs(), kn[b].abs()).amax(-1) * dim ** -0.5
        cap = scores.get("softcap", 0.0)
        if cap:
            s = cap * torch.tanh(s / cap)
        size = s.abs().amax(-1)
        if scores.get("slopes") is not None:
            s = s - scores["slopes"].double().view(hk, -1, 1) * distance[:, None, None]
        s = s.masked_fill(((distance < 0) | (distance >= (scores.get("window") or keys)))[:, None, None], -math.inf)
        z = torch.logsumexp(s, -1)
        w = torch.exp(s - z[..., None])
        want["out"].append(torch.einsum("shgn,nhd->shgd", w, vn[b]))
        want["spread"].append(torch.einsum("shgn,nhd->shgd", w, vn[b].abs()))
        want["top"].append(w.amax(-1)[..., None] * vn[b].abs().sum(0)[None, :, None])
        want["lse"].append(z)
        want["reach"].append(reach)
        want["score"].append(size)
    want = {n: torch.stack(x).reshape(batch * slots, hq, *x[0].shape[3:]) for n, x in want.items()}
    return out.double().view(batch * slots, hq, dim), lse.double(), want


def check(dtype, eight, got, lse, want, keys, dim, cap=0.0, slack=0.0):
    """A score's fp32 sum of dim products, its scalings and the exponent's argument: (dim + 8) e of sum |q k|.  A capped one is
    off by 16 e of itself and, next to a cap of up to 256 in units of log2 (178), of the cap.  A weight is rounded to the
    type: u (f16 over 8-bit caches, no more than that)."""
    score = (dim + 8) * E * (want["reach"] + 16) + (16 * E * min(cap, 178.0) + 40 * E * want["score"] if cap else 0.0)
    off = (U[dtype] + 2 * score[..., None] + (keys + 64) * E) * want["spread"] + U[dtype] * want["out"].abs() + slack + 2.0 ** -24
    assert torch.all((lse - want["lse"]).abs() <= score + (keys + 16) * E + 2 * E * want["lse"].abs())
    assert torch.all((got - want["out"]).abs() <= off)


CAPS = [2.2e4, 2.4e4, 1e6, 1e9, 8e37]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype,eight,slots,hq,hk,dim", [
    ("bf16", False, 1, 4, 2, 128), ("f16", False, 19, 4, 1, 64), ("bf16", False, 61, 8, 2, 128), ("f16", False, 61, 4, 1, 128),
    ("bf16", True, 1, 4, 2, 128), ("f16", True, 3, 4, 1, 64), ("bf16", True, 19, 4, 2, 64), ("f16", True, 61, 8, 2, 128)])
def test_a_cap_far_above_the_scores_changes_next_to_nothing(cap, dtype, eight, slots, hq, hk, dim):
    gen = torch.Generator(device="cuda").manual_seed(slots + dim)
    q = torch.randn((2, slots, hq, dim), generator=gen, device="cuda") * 6
    k, v = (torch.randn((2, 700 + slots, hk, dim), generator=gen, device="cuda") for _ in range(2))
    got, lse, want = attend(dtype, eight, q, k, v, softcap=cap)
    check(dtype, eight, got, lse, want, 700 + slots, dim, cap)


@pytest.mark.parametrize("more", [dict(prefix=300), dict(prefix=300, window=500), dict(window=90), dict(prefix=40, slopes=0.2)],
                         ids=lambda m: "-".join(m))
@pytest.mark.parametrize("cap", [300.0, 1e6])
@pytest.mark.parametrize("dtype,eight,slots,hq,hk,dim", [
    ("bf16", False, 2, 4, 2, 64), ("f16", False, 61, 8, 2, 128), ("f16", True, 1, 4, 1, 128), ("bf16", True, 40, 8, 2, 64)])
def test_wide_caps_with_all_else(cap, more, dtype, eight, slots, hq, hk, dim):
    gen = torch.Generator(device="cuda").manual_seed(slots + dim)
    q = torch.randn((3, slots, hq, dim), generator=gen, device="cuda") * 6
    k, v = (torch.randn((3, 800 + slots, hk, dim), generator=gen, device="cuda") for _ in range(2))
    more = dict(more)
    if "slopes" in more:
        more["slopes"] = torch.full((hq,), more["slopes"], device="cuda")
    got, lse, want = attend(dtype, eight, q, k, v, softcap=cap, **more)
    # the bias adds 4 e of itself to a score: at most 0.2 times the keys, where a weight counts far less
    check(dtype, eight, got, lse, want, 800 + slots, dim, cap, slack=2 * 4 * E * 0.2 * 900 * want["spread"] if "slopes" in more else 0.0)


@pytest.mark.parametrize("cap", [30.0, 150.0, 400.0, 3000.0, 2e4])
@pytest.mark.parametrize("dtype,eight,slots,hq,hk,dim", [
    ("f16", False, 19, 4, 1, 64), ("f16", False, 61, 8, 2, 128), ("f16", True, 4, 4, 1, 64), ("f16", True, 61, 8, 2, 128),
    ("bf16", True, 61, 4, 1, 64)])
def test_rows_of_small_scores_beside_rows_at_the_cap(cap, dtype, eight, slots, hq, hk, dim):
    """Every other row's scores come near the cap, those beside it are of about 3: none loses by its neighbour."""
    gen = torch.Generator(device="cuda").manual_seed(slots + dim)
    if dtype == "bf16":                 # whose queries may be larger
        cap *= 50
    q = torch.randn((2, slots, hq, dim), generator=gen, device="cuda") * 3
    k, v = (torch.randn((2, 700 + slots, hk, dim), generator=gen, device="cuda") for _ in range(2))
    q[:, ::2] *= cap / 9
    got, lse, want = attend(dtype, eight, q, k, v, softcap=cap)
    check(dtype, eight, got, lse, want, 700 + slots, dim, cap)


@pytest.mark.parametrize("gap", [12.0, 16.0, 18.0, 20.0])
@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("dtype,eight", [("bf16", True), ("f16", True), ("f16", False), ("bf16", False)])
@pytest.mark.parametrize("batch,slots,prefix,hq,hk,dim", [
    (80, 1, 0, 8, 2, 64), (80, 4, 0, 4, 2, 128), (80, 9, 0, 8, 2, 64), (80, 40, 0, 8, 2, 128),     # an item whole, or nearly
    (1, 61, 0, 8, 2, 128), (40, 2, 3000, 8, 4, 128), (20, 61, 3000, 4, 1, 64)])
def test_a_first_key_that_outweighs_the_others(gap, spread, dtype, eight, batch, slots, prefix, hq, hk, dim):
    """Key 0 scores `gap` above thousands of others (in logarithms of weights), all alike or spread, and its value is zero, so
    the result is made of weights that are small next to the largest.  f16 weights (8-bit caches, f16 models) that are
    subnormal are off by 2^-25 at most, with the first maximum's at 2^6: 2^-31 of the row's largest."""
    keys = 4000 + slots
    gen = torch.Generator(device="cuda").manual_seed(slots + dim)
    q, k, v = (torch.randn(s, generator=gen, device="cuda") for s in ((batch, slots, hq, dim), (batch, keys, hk, dim), (batch, keys, hk, dim)))
    q[..., 0], k[..., 0] = 8.0, 0.0
    k *= spread
    k[:, 0] = 0.0
    k[:, 0, :, 0] = gap * dim ** 0.5 / 8
    v = v + 1
    v[:, 0] = 0.0
    got, lse, want = attend(dtype, eight, q, k, v, prefix)
    half = dtype == "f16" or eight
    check(dtype, eight, got, lse, want, keys, dim, slack=2.0 ** -31 * want["top"] if half else 0.0)


@pytest.mark.parametrize("slope", [0.3, 50.0, 1e37])
@pytest.mark.parametrize("prefix,own", [(5, 0), (5, 3), (130, 1), (100, 300)])
@pytest.mark.parametrize("dtype,eight,slots,hq,hk,dim", [
    ("bf16", False, 1, 4, 2, 128), ("f16", False, 20, 4, 2, 64), ("bf16", True, 40, 4, 1, 128), ("f16", True, 2, 4, 1, 64)])
def test_slopes_behind_a_prefix_that_ends_inside_a_block(slope, prefix, own, dtype, eight, slots, hq, hk, dim):
    """However steep, a slope leaves a row its own key."""
    keys = prefix + own + slots
    gen = torch.Generator(device="cuda").manual_seed(keys + dim)
    q, k, v = (torch.randn(s, generator=gen, device="cuda") for s in ((1, slots, hq, dim), (1, keys, hk, dim), (1, keys, hk, dim)))
    got, lse, want = attend(dtype, eight, q, k, v, prefix, slopes=torch.full((hq,), slope, device="cuda"))
    check(dtype, eight, got, lse, want, keys, dim)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_what_is_read_back_is_the_fp32_product_rounded_to_the_type(dtype):
    """Bit for bit: every code under scales of every last bit, products beyond the type's range and below its smallest among
    them."""
    heads = 300
    gen = torch.Generator().manual_seed(5)
    scale = torch.exp2(torch.rand(heads, generator=gen) * 60 - 40)
    codes = torch.arange(256, dtype=torch.uint8)
    cache = codes.view(1, 1, 4, 64).repeat(1, heads, 2, 1).cuda()       # one page of 8 tokens
    kv = g.GraftKV(g.graft_kv_default_config(heads, heads, 64, 8, 1, 1, 1, GDT[dtype], cache="e4m3"))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.empty((4, heads * 64), dtype=DT[dtype], device="cuda") for _ in range(2)]
    kv.read(1, 4, cache, cache, zero.view(1, 1), zero, zero + 4, *outs, k_scale=scale.cuda(), v_scale=scale.cuda())
    assert kv.sync() == 0
    number = codes.view(E4M3).float()
    want = (scale[:, None] * number).to(DT[dtype]).view(heads, 4, 64).transpose(0, 1)
    finite = ~torch.isnan(want)
    assert finite.sum() == heads * 254
    for o in outs:
        got = o.cpu().view(4, heads, 64)
        assert torch.equal(torch.isnan(got), ~finite)
        assert torch.equal(got.view(torch.int16)[finite], want.contiguous().view(torch.int16)[finite])
