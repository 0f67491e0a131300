"""The operators together: a small target decoded with trees emits what it would emit token by token.

Every emitted token is checked with the model run plainly in fp32 over the whole sequence before it (no cache, no tree):
its ruled logit must be within the activations' bf16 noise of the largest.  The logits have a spread of about 4; a chain of
some ten roundings of relative size 2^-9 gives each about 0.03, so the two that compare differ by less than 0.4 (over 9 of
those).  A key at a wrong place, a wrong position or a wrong mask moves logits by their spread."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.cuda.set_device(0)


def plain_logits(m, tokens):
    """Logits after each token of one sequence, in fp32."""
    x = m.embed[tokens].float()
    n, d = len(tokens), m.head_dim
    rope = m.rope(n)
    cos, sin = rope[:, None, :d // 2], rope[:, None, d // 2:]

    def turn(y):
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    norm = lambda y: y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    for w, o in zip(m.qkv, m.out):
        q, k, v = (norm(x) @ w.float()).split([m.q_heads * d, m.kv_heads * d, m.kv_heads * d], 1)
        q, k, v = turn(q.view(n, -1, d)), turn(k.view(n, -1, d)), v.view(n, -1, d)
        k, v = (y.repeat_interleave(m.q_heads // m.kv_heads, 1) for y in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device=s.device).triu(1), -float("inf"))
        x = x + torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(n, -1) @ o.float()
    return norm(x) @ m.head.float()


@pytest.mark.parametrize("prefix_len,lengths", [(0, [5]), (150, [40, 1, 90]), (16, [70, 3])])
def test_tree_decoding_emits_the_targets_own_tokens(prefix_len, lengths):
    from workloads.target_model import TargetLoop, ToyTarget
    torch.manual_seed(prefix_len)
    m = ToyTarget(seed=prefix_len + 1)
    prefix = torch.randint(0, m.vocab, (prefix_len,)).tolist()
    prompts = [torch.randint(0, m.vocab, (n,)).tolist() for n in lengths]
    penalty = torch.tensor([[1.2, 0.3, 0.1], [1.0, 0.0, 0.0], [0.9, -0.2, 0.5]][:len(prompts)], device="cuda")
    # after an even token only even tokens, after an odd one everything
    words = torch.full((2, (m.vocab + 31) // 32), -1, dtype=torch.int32, device="cuda")
    words[0] = 0x55555555
    grammar_of = (torch.arange(m.vocab, device="cuda", dtype=torch.int32) % 2)
    loop = TargetLoop(m, prefix, prompts, penalty=penalty, grammar=words, grammar_of=grammar_of)
    accepted = sum(sum(loop.step()) for _ in range(10))
    assert accepted > 0                       # paths of more than the root were written again at contiguous places
    for b, p in enumerate(prompts):
        seq = p + loop.emitted[b]
        assert loop.hist[b, :len(seq)].tolist() == seq and int(loop.ctx[b]) == len(seq) - 1
        logits = plain_logits(m, torch.tensor(prefix + seq, device="cuda"))[len(prefix):]
        r, f, pres = penalty[b].tolist()
        for i, t in enumerate(loop.emitted[b]):
            before = seq[:len(p) + i]
            x = logits[len(before) - 1].clone()
            n = torch.bincount(torch.tensor(before[len(p):], device="cuda", dtype=torch.int64), minlength=m.vocab)
            seen = n > 0
            seen[torch.tensor(p, device="cuda")] = True
            x = torch.where(seen, torch.where(x > 0, x / r, x * r), x) - f * n - pres * (n > 0)
            if before[-1] % 2 == 0:
                x[1::2] = -float("inf")
                assert t % 2 == 0
            assert x[t] >= x.max() - 0.4, (b, i, t)


def test_the_longest_request_is_refused_before_its_pages_end():
    """The bound that the loop passes follows its requests; one that has outgrown its pages is refused, and nothing ran."""
    from workloads.target_model import TargetLoop, ToyTarget
    loop = TargetLoop(ToyTarget(seed=3), [], [list(range(20)), [5]], longest=24)
    steps = 0
    with pytest.raises(ValueError, match="24 tokens"):
        for steps in range(30):
            loop.step()
            assert loop.ctx.tolist() == loop.held
    assert steps > 0 and loop.kv.sync() == 0 and max(loop.held) <= 24 + loop.S
