"""A small target model around the draft tree, on the paged cache.

The verification step needs the target's logits of every tree slot.  This is
how a model produces them with the library: per layer the slots' queries and
keys are rotated and their keys and values appended to the paged cache
(``GraftKV.append``), the slots attend over the shared prompt, their request's
context and their own path (``GraftKV.attend``); the logits pass the rules
(``Graft.process_logits``), the tree is verified (``Graft.verify_update``), and
the accepted slots' keys and values are written again at contiguous places
(``GraftKV.append`` with ``rows``).  A model may cap its scores, look back
over a window, bias scores by the distance, or rotate by positions of three
axes; the loop may hold the cache in 8 bits.  Weights are random; ``python -m
workloads.target_model`` decodes a few steps and prints what they accept.
"""
from __future__ import annotations

import torch

import hybrid_draft_tree_gb300 as g


class ToyTarget:
    """Random weights: embedding, `layers` of attention with a residual, head.  The residual outweighs the attention, so a
    token says much about its successor, as in text, and retrieved trees are accepted now and then."""

    def __init__(self, vocab=1000, layers=2, q_heads=8, kv_heads=2, head_dim=64, hidden=256, device="cuda", seed=0, softcap=0.0,
                 window=0, alibi=False, axes=False):
        """window: of every other layer, from the first on, as in models that alternate; alibi: scores fall with the
        distance; axes: pairs turn by three positions (see positions_of)."""
        self.softcap, self.window, self.axes = softcap, window, axes
        self.slopes = 2.0 ** (-8.0 * torch.arange(1, q_heads + 1, device=device) / q_heads) if alibi else None
        gen = torch.Generator(device=device).manual_seed(seed)
        self.vocab, self.layers, self.q_heads, self.kv_heads, self.head_dim = vocab, layers, q_heads, kv_heads, head_dim
        widths = (q_heads + 2 * kv_heads) * head_dim

        def weight(rows, cols, scale=1.0):
            return (torch.randn((rows, cols), generator=gen, device=device) * scale * rows ** -0.5).bfloat16()
        self.embed = torch.randn((vocab, hidden), generator=gen, device=device).bfloat16()
        self.qkv = [weight(hidden, widths, 1.5) for _ in range(layers)]
        self.out = [weight(q_heads * head_dim, hidden, 0.7) for _ in range(layers)]
        self.head = weight(hidden, vocab, 4.0)

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)

    def pair_axis(self):
        """The axis whose position turns a pair: time for the first quarter, then height and width."""
        half = self.head_dim // 2
        return [0 if i < half // 4 else 1 + i % 2 for i in range(half)]

    @staticmethod
    def positions_of(place):
        """Positions [3, ...] of the token at a place of the sequence, as if it were read as an image of 7 columns."""
        return torch.stack([place, place // 7, place % 7])

    def scores(self, layer):
        return dict(softcap=self.softcap, window=self.window if layer % 2 == 0 else 0, slopes=self.slopes)

    def rope(self, positions):
        angle = torch.arange(positions, device=self.embed.device)[:, None] * 10000.0 ** (
            -torch.arange(0, self.head_dim, 2, device=self.embed.device) / self.head_dim)
        return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def accepted_rows(tok, parent, accept_len, out_tokens):
    """The slots of each request's accepted path, the root first, then -1: int32 [batch, S].  The path is the one whose
    tokens were emitted; where siblings repeat a token several are, and it is the one that ends in the lowest slot."""
    batch, S = tok.shape
    rows = torch.full((batch, S), -1, dtype=torch.int32, device=tok.device)
    rows[:, 0] = 0
    slot, above = torch.arange(S, device=tok.device), parent.long().clamp(min=0)
    most = int(accept_len.max())
    level = (slot == 0).expand(batch, S)              # the slots that paths of the emitted tokens have reached
    for d in range(most):
        below = level.gather(1, above) & (tok == out_tokens[:, d:d + 1]) & (slot > 0)
        level = torch.where((d < accept_len)[:, None], below, level)
    end = torch.where(level, slot, S).amin(1)
    for d in range(most, 0, -1):
        on = d <= accept_len
        rows[:, d] = torch.where(on, end, -1)
        end = torch.where(on, above.gather(1, end.clamp(max=S - 1)[:, None])[:, 0], end)
    return rows


class TargetLoop:
    """Decodes `prompts` (lists of tokens behind the shared `prefix`) with trees retrieved from the continuation matrix.

    Trees are all retrieval (the fixed split with no draft slots), so no drafter is needed; a drafter's trees go the
    same way.  `penalty` [batch, 3] and `grammar` / `grammar_of` (the row of a token's successors) are the rules.  `cache`
    "e4m3" holds keys and values in 8 bits, with `scales` (k_scale, v_scale: float32 [kv_heads])."""

    def __init__(self, model, prefix, prompts, longest=512, page=16, penalty=None, grammar=None, grammar_of=None, cache=None,
                 scales=None):
        dev = model.embed.device
        self.m, self.B, self.page = model, len(prompts), page
        self.penalty, self.grammar, self.grammar_of = penalty, grammar, grammar_of
        self.eng = g.Graft(g.graft_default_config(model.vocab, self.B, g.GRAFT_MODE_CHECKPOINT, g.GRAFT_BF16, ablation=2,
                                                  fixed_draft=0))
        self.S = self.eng.S
        # the matrix starts from what the model says of each token alone
        every = torch.arange(model.vocab, dtype=torch.int32, device=dev)
        self.eng.warmup(every, model.norm(model.embed) @ model.head)
        own, pre = -(-(longest + self.S) // page), -(-len(prefix) // page)
        pages = self.B * own + pre
        self.kv = g.GraftKV(g.graft_kv_default_config(model.q_heads, model.kv_heads, model.head_dim, page, pages, max(self.B, 1),
                                                      64, cache=cache))
        self.scales = {} if scales is None else dict(k_scale=scales[0], v_scale=scales[1])
        if model.axes:
            self.kv.set_axes(model.pair_axis())
        self.prefix_pages = torch.arange(pre, dtype=torch.int32, device=dev)
        self.table = torch.arange(pre, pages, dtype=torch.int32, device=dev).view(self.B, own)
        self.longest, self.prefix_len = longest, len(prefix)
        shape = (pages, model.kv_heads, page, model.head_dim)
        kind = torch.bfloat16 if cache is None else torch.float8_e4m3fn
        self.caches = [tuple(torch.empty(shape, dtype=kind, device=dev) for _ in range(2)) for _ in range(model.layers)]
        self.rope = model.rope(len(prefix) + longest + self.S)
        self.ctx = torch.zeros(self.B, dtype=torch.int32, device=dev)
        # the prefix is a request of its own whose pages everybody reads; then each prompt but its last token
        if len(prefix):
            self._prefill(torch.tensor([prefix], dtype=torch.int32, device=dev), self.prefix_pages.view(1, -1), 0,
                          torch.zeros(1, dtype=torch.int32, device=dev))
        most = max(len(p) for p in prompts)
        self.hist = torch.zeros((self.B, longest + self.S + 1), dtype=torch.int32, device=dev)
        for b, p in enumerate(prompts):
            self.hist[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
            if len(p) > 1:
                self._prefill(self.hist[b:b + 1, :len(p) - 1].contiguous(), self.table[b:b + 1], self.prefix_len,
                              self.ctx[b:b + 1])
        self.hist_len = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
        self.prompt_len = self.hist_len.clone()
        self.ctx = self.hist_len - 1
        self.emitted = [[] for _ in prompts]
        self.held = [len(p) - 1 for p in prompts]      # the host's copy of ctx: its largest bounds the attention's work
        assert most <= longest

    def _prefill(self, tokens, table, prefix_len, ctx):
        """One request's tokens, 64 at a time, each seeing those before it."""
        for at in range(0, tokens.shape[1], 64):
            part = tokens[:, at:at + 64].contiguous()
            self._forward(part, None, None, table.contiguous(), prefix_len, ctx + at, at)

    def _positions(self, slots, pos, prefix_len, ctx):
        """What append takes of them: nothing, or the slots' positions on three axes."""
        if not self.m.axes:
            return None
        depth = torch.arange(slots, device=ctx.device).expand(len(ctx), slots) if pos is None else pos.clamp(min=0)
        return self.m.positions_of(prefix_len + ctx[:, None] + depth).int().contiguous()

    def _forward(self, tok, pos, mask, table, prefix_len, ctx, max_ctx):
        """Logits [batch * slots, V] of the slots, and the layers' k and v rows."""
        m, (batch, slots) = self.m, tok.shape
        x = m.embed[tok.clamp(min=0).long().view(-1)]
        widths = [m.q_heads * m.head_dim, m.kv_heads * m.head_dim, m.kv_heads * m.head_dim]
        q_rot, attn = (torch.zeros((batch * slots, widths[0]), dtype=x.dtype, device=x.device) for _ in range(2))
        kept, positions = [], self._positions(slots, pos, prefix_len, ctx)
        for layer, (kc, vc) in enumerate(self.caches):
            q, k, v = (m.norm(x) @ m.qkv[layer]).split(widths, 1)
            self.kv.append(batch, slots, q, k, v, self.rope, table, ctx, kc, vc, q_rot, prefix_len=prefix_len, pos=pos,
                           positions=positions, **self.scales)
            self.kv.attend(batch, slots, q_rot, kc, vc, table, ctx, max_ctx, attn,
                           prefix_pages=self.prefix_pages if prefix_len else None, prefix_len=prefix_len, tree_mask=mask,
                           **m.scores(layer), **self.scales)
            x = x + attn @ m.out[layer]
            kept.append((k, v))
        return m.norm(x) @ m.head, kept

    def step(self):
        """One decode step of every request; returns the accepted lengths."""
        if max(self.held) > self.longest:
            raise ValueError(f"a request has passed the {self.longest} tokens that the pages were laid out for")
        B, S, eng, dev = self.B, self.S, self.eng, self.hist.device
        t = g.TreeBuffers(B, S, dev)
        root = self.hist.gather(1, (self.hist_len - 1).long()[:, None]).view(-1)
        none = torch.zeros((B, 0), device=dev)
        eng.assemble(B, root, none.int(), none.short(), none.float(), t.tok, t.parent, t.pos, t.mask, t.info)
        logits, kept = self._forward(t.tok, t.pos, t.mask, self.table, self.prefix_len, self.ctx, max(self.held))
        rules = {}
        if self.grammar is not None:
            rules = dict(grammar=self.grammar, grammar_row=self.grammar_of[t.tok.clamp(min=0).long()].contiguous())
        ruled = torch.empty_like(logits)
        eng.process_logits(B, S, logits, ruled, tree_tok=t.tok, tree_mask=t.mask, hist=self.hist, hist_len=self.hist_len,
                           prompt_len=self.prompt_len, penalty=self.penalty, **rules)
        eng.verify_update(B, t.tok, t.parent, t.pos, t.mask, ruled, t.accept_len, t.out_tokens)
        rows = accepted_rows(t.tok, t.parent, t.accept_len, t.out_tokens)
        positions = self._positions(S, t.pos, self.prefix_len, self.ctx)
        for (kc, vc), (k, v) in zip(self.caches, kept):
            self.kv.append(B, S, None, k, v, self.rope, self.table, self.ctx, kc, vc, None, prefix_len=self.prefix_len,
                           pos=t.pos, rows=rows, positions=positions, **self.scales)
        accepted = t.accept_len.tolist()
        for b, n in enumerate(accepted):
            new = t.out_tokens[b, :n + 1]
            at = int(self.hist_len[b])
            self.hist[b, at:at + n + 1] = new
            self.emitted[b] += new.tolist()
            self.held[b] += n + 1
        self.hist_len += t.accept_len + 1
        self.ctx += t.accept_len + 1
        assert eng.sync() == 0 and self.kv.sync() == 0
        return accepted


def main():
    torch.manual_seed(0)
    model = ToyTarget()
    prefix = torch.randint(0, model.vocab, (150,)).tolist()
    prompts = [torch.randint(0, model.vocab, (n,)).tolist() for n in (40, 7, 90)]
    penalty = torch.tensor([[1.05, 0.1, 0.0]] * len(prompts), device="cuda")
    loop = TargetLoop(model, prefix, prompts, penalty=penalty)
    for step in range(8):
        print(f"step {step}: accepted {loop.step()} draft tokens, context {loop.ctx.tolist()}")
    for b, e in enumerate(loop.emitted):
        print(f"request {b}: {e}")


if __name__ == "__main__":
    main()
