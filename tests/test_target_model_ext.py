"""The small target over an 8-bit cache, with capped, windowed and distance-biased scores and with positions of three axes:
trees decoded with the library emit what the model would emit token by token.

Every emitted token is checked with the model run plainly in fp32 over the whole sequence before it (no cache, no tree), keys
and values rounded to e4m3 as they are in the cache: its ruled logit must be within the activations' noise of the largest.
The logits have a spread of about 4; a chain of some ten roundings of relative size 2^-9 gives each about 0.03, so the two that
compare differ by less than 0.4 (over 9 of those).  In 8 bits a value whose rotation or projection was rounded to the other side
of a border of two numbers is 2^-3 of itself off; with bf16 rows (steps of 2^-8 within numbers 2^-3 apart) that is one element in
some 30, which adds a noise of 2^-3 / sqrt(12 * 30), 0.7 of 2^-7, to each key's score and each value: about twice the chain's
own.  A key at a wrong place, a wrong position or a wrong mask moves logits by their spread."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.cuda.set_device(0)


def plain_logits(m, tokens, scales):
    """Logits after each token of one sequence, in fp32."""
    x = m.embed[tokens].float()
    n, d = len(tokens), m.head_dim
    place = torch.arange(n, device=x.device)
    rope, half = m.rope(n), d // 2
    at = place[:, None].expand(n, half)
    if m.axes:
        at = m.positions_of(place)[m.pair_axis()].t()
    pair = torch.arange(half, device=x.device)
    cos, sin = rope[at, pair][:, None], rope[at, pair + half][:, None]

    def turn(y):
        a, b = y[..., :half], y[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    def held(y, scale):
        if scale is None:
            return y
        return (y / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float() * scale[:, None]
    norm = lambda y: y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    distance = place[:, None] - place
    for layer, (w, o) in enumerate(zip(m.qkv, m.out)):
        q, k, v = (norm(x) @ w.float()).split([m.q_heads * d, m.kv_heads * d, m.kv_heads * d], 1)
        q, k, v = turn(q.view(n, -1, d)), held(turn(k.view(n, -1, d)), scales and scales[0]), held(v.view(n, -1, d), scales and scales[1])
        k, v = (y.repeat_interleave(m.q_heads // m.kv_heads, 1) for y in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        shape = m.scores(layer)
        if shape["softcap"]:
            s = shape["softcap"] * torch.tanh(s / shape["softcap"])
        if shape["slopes"] is not None:
            s = s - shape["slopes"][:, None, None] * distance
        s.masked_fill_((distance < 0) | (distance >= (shape["window"] or n)), -float("inf"))
        x = x + torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(n, -1) @ o.float()
    return norm(x) @ m.head.float()


@pytest.mark.parametrize("prefix_len,lengths,cache,shape", [
    (150, [40, 1, 90], "e4m3", {}),
    (0, [70, 5], "e4m3", dict(softcap=2.0, window=40)),
    (150, [40, 1], None, dict(softcap=2.0, window=33)),
    (16, [70, 3], None, dict(alibi=True)),
    (20, [9, 60], None, dict(axes=True)),
    (150, [40, 7], "e4m3", dict(axes=True, window=100, alibi=True)),
])
def test_tree_decoding_emits_the_targets_own_tokens(prefix_len, lengths, cache, shape):
    from workloads.target_model import TargetLoop, ToyTarget
    torch.manual_seed(prefix_len)
    m = ToyTarget(seed=prefix_len + 1, **shape)
    prefix = torch.randint(0, m.vocab, (prefix_len,)).tolist()
    prompts = [torch.randint(0, m.vocab, (n,)).tolist() for n in lengths]
    penalty = torch.tensor([[1.2, 0.3, 0.1], [1.0, 0.0, 0.0], [0.9, -0.2, 0.5]][:len(prompts)], device="cuda")
    scales = (torch.tensor([0.02, 0.03], device="cuda"), torch.tensor([0.015, 0.02], device="cuda")) if cache else None
    loop = TargetLoop(m, prefix, prompts, penalty=penalty, cache=cache, scales=scales)
    accepted = sum(sum(loop.step()) for _ in range(10))
    assert accepted > 0                       # paths of more than the root were written again at contiguous places
    for b, p in enumerate(prompts):
        seq = p + loop.emitted[b]
        assert loop.hist[b, :len(seq)].tolist() == seq and int(loop.ctx[b]) == len(seq) - 1
        logits = plain_logits(m, torch.tensor(prefix + seq, device="cuda"), scales)[len(prefix):]
        r, f, pres = penalty[b].tolist()
        for i, t in enumerate(loop.emitted[b]):
            before = seq[:len(p) + i]
            x = logits[len(before) - 1].clone()
            n = torch.bincount(torch.tensor(before[len(p):], device="cuda", dtype=torch.int64), minlength=m.vocab)
            seen = n > 0
            seen[torch.tensor(p, device="cuda")] = True
            x = torch.where(seen, torch.where(x > 0, x / r, x * r), x) - f * n - pres * (n > 0)
            # in 8 bits the noise is some three times the chain's own
            assert x[t] >= x.max() - (1.2 if cache else 0.4), (b, i, t)
