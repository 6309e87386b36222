"""One request loop around drafted blocks: draft, score over the paged cache, verify, cut back.

A small random target model (embedding, one attention layer over the cache, unembedding) decodes
N requests that share a prompt.  Every step

  1. the refinement drafts a block per request            xp_jacobi_refine
     (or tokens are drawn from its logits, which the
     verification then needs)                             xp_latent_pass, xp_refine_logits
  2. the cache takes pages for the block                  xp_cache_resize
  3. the block's keys and values go in                    xp_cache_append
  4. the target attends for all B slots at once,
     the shared prompt read once for the batch            xp_prefix_attention
  5. the drafts are verified, one token is drawn          xp_verify_drafts
     and what was emitted is scored, if asked for         xp_token_logprobs
  6. what was not accepted leaves the cache               xp_cache_resize

(the cache may be one of 8 or 4 bits: the calls are the same) and at the end one request is continued twice (xp_cache_fork), another dropped, and the pool
packed (xp_cache_compact).

    python -m examples.verify_step
"""
from __future__ import annotations

import math

import torch

from jacobi_speculative_decode_gb300 import xp


class Target:
    """Next token mostly a fixed successor of the last one, bent by attention over what came before."""

    def __init__(self, vocab=512, heads=8, kv_heads=2, dim=64, dtype=torch.float32, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.vocab, self.heads, self.kv_heads, self.dim, self.dtype = vocab, heads, kv_heads, dim, dtype
        width = heads * dim

        def weight(*shape):
            return (torch.randn(shape, generator=g) / math.sqrt(shape[0])).to(dtype).cuda()

        self.embed = torch.randn(vocab, width, generator=g).to(dtype).cuda()
        self.successor = torch.randperm(vocab, generator=g).cuda()
        self.unembed = torch.empty(width, vocab, dtype=dtype, device="cuda")
        self.unembed[:, self.successor] = self.embed.t() * (8.0 / width)
        self.wq, self.wo = weight(width, width) * 2, weight(width, width) * 16
        self.wk, self.wv = weight(width, kv_heads * dim), weight(width, kv_heads * dim)

    def qkv(self, tokens):
        x = self.embed[tokens]
        shape = tokens.shape + (-1, self.dim)
        return x, (x @ self.wq).view(shape), (x @ self.wk).view(shape), (x @ self.wv).view(shape)

    def logits(self, x, attended):
        return (x + attended.reshape(x.shape) @ self.wo) @ self.unembed


class Drafter:
    """A refinement head of random weights; its base logits name the target's usual successors."""

    def __init__(self, target, block, requests, seed=1):
        g = torch.Generator().manual_seed(seed)
        V, self.hidden, r, H, B = target.vocab, 64, 32, 64, block
        shapes = dict(w1=(V, r), down_h=(r, self.hidden), down_g=(r, self.hidden), in_proj=(r, 3 * r),
                      mix_L=(r, B, B), w_gate=(H, r), w_up=(H, r), w_down=(r, H), w2=(V, r))
        weights = {k: (torch.randn(s, generator=g) * 0.1).to(target.dtype).cuda() for k, s in shapes.items()}
        dtype = "bf16" if target.dtype == torch.bfloat16 else "f32"
        self.head = xp.Head(dict(V=V, hidden=self.hidden, r=r, H=H, B=B), weights, dtype, requests)
        self.target, self.B = target, B
        self.ws, self.verify_ws = self.head.workspace(requests), self.head.verify_workspace(requests)
        self.blk = torch.empty(requests, B, dtype=torch.int64, device="cuda")

    def draft(self, anchor, before, passes=2):
        """Blocks [N, B] that continue `anchor` (whose predecessor is `before`)."""
        N, B, V = anchor.numel(), self.B, self.target.vocab
        base = torch.zeros(N, B - 1, V, dtype=self.target.dtype, device="cuda")
        token = anchor
        for b in range(B - 1):
            token = self.target.successor[token]
            base[torch.arange(N), b, token] = 6.0
        h = torch.zeros(N, B, self.hidden, dtype=self.target.dtype, device="cuda")
        xp.xp_jacobi_refine(self.head.handle, base, (B - 1) * V, V, h, anchor, before, N, passes, 0,
                            self.blk, self.ws)
        self.base, self.h = base, h
        return self.blk

    def sample(self, anchor, before, heat, generator, passes=2):
        """Blocks whose drafts are drawn from the refinement's distribution at temperatures `heat` [N]
        (their argmax at 0), and the logits [N*(B-1), V] of that distribution."""
        N, B, V, r = anchor.numel(), self.B, self.target.vocab, self.head.r
        blk = self.draft(anchor, before, passes)
        xh = torch.empty(N, B, r, device="cuda")
        xp.xp_hidden_cache(self.head.handle, self.h, N, xh, self.ws)
        lat = torch.empty(N, B - 1, r, dtype=self.target.dtype, device="cuda")
        xp.xp_latent_pass(self.head.handle, blk, before, xh, N, lat)
        logits = torch.empty(N * (B - 1), V, device="cuda")
        xp.xp_refine_logits(self.head.handle, lat, self.base, (B - 1) * V, V, N, logits, V)
        race = torch.empty(N, B - 1, V).exponential_(generator=generator).clamp_(min=1e-20).cuda()
        hot = torch.where(heat > 0, heat, 1.0)[:, None, None]
        drawn = logits.view(N, B - 1, V) / hot - torch.log(race) * (heat > 0)[:, None, None]
        blk[:, 1:] = drawn.argmax(-1)
        return blk, logits


def run(requests=5, block=6, steps=6, prompt_len=75, page=16, temperature=0.0, dtype=torch.float32,
        seed=0, sampled=False, bits=0, scores=None, top=3):
    """Decode `requests` continuations of one prompt, from greedy drafts or (sampled) from drafts drawn
    from the refinement's logits, over a cache of the target's type or (bits, 8 or 4; bf16 targets) a quantised
    one.  Returns (target, prompt, first tokens, tokens emitted by each request, drafts accepted, drafts made).
    scores: a list that receives, for every step, the logits, the tokens emitted and their logprob, entropy,
    rank and `top` alternatives."""
    target = Target(dtype=dtype, seed=seed)
    drafter = Drafter(target, block, requests)
    g = torch.Generator().manual_seed(seed + 7)
    N, B, V = requests, block, target.vocab
    H, D = target.kv_heads, target.dim
    int32 = dict(dtype=torch.int32, device="cuda")
    width = -(-(steps + 1) * B // page)
    prompt_pages = -(-prompt_len // page)
    pages = prompt_pages + (N + 2) * width
    if bits:
        k, v = (xp.QuantCache.pool(1, pages, page, H, D, bits) for _ in range(2))
        cache = xp.QuantCache(k, v, page, D, bits)
    else:
        k, v = (torch.empty(1, pages, page, H, D, dtype=dtype, device="cuda") for _ in range(2))
        cache = xp.Cache(k, v)

    # row 0 of the table is the shared prompt, the requests' tails follow
    table = torch.full((N + 1, max(width, prompt_pages)), -1, **int32)
    lens, refs = torch.zeros(N + 1, **int32), torch.zeros(pages, **int32)
    prompt = torch.randint(0, V, (prompt_len,), generator=g).cuda()
    first = torch.zeros(N + 1, **int32)
    first[0] = prompt_len
    xp.xp_cache_resize(cache.handle, table, lens, first, refs, table, lens, refs)
    _, _, pk, pv = target.qkv(prompt[None])
    xp.xp_cache_append(cache.handle, 0, pk, pv, table[:1], lens[:1])

    anchor = torch.randint(0, V, (N,), generator=g).cuda()
    start, before = anchor.clone(), prompt[-1].repeat(N)
    heat = torch.full((N,), float(temperature), device="cuda")
    tokens = torch.empty(N, B, dtype=torch.int64, device="cuda")
    counts = torch.empty(N, **int32)
    out = torch.empty(N, B, target.heads, D, dtype=dtype, device="cuda")
    emitted, accepted = [[] for _ in range(N)], 0
    tails, lengths = table[1:], lens[1:]
    for _ in range(steps):
        blk, draft = drafter.sample(anchor, before, heat, g) if sampled \
            else (drafter.draft(anchor, before), None)
        kept = lens.clone()
        want = kept + B
        want[0] = prompt_len
        xp.xp_cache_resize(cache.handle, table, lens, want, refs, table, lens, refs)
        x, q, nk, nv = target.qkv(blk)
        xp.xp_cache_append(cache.handle, 0, nk, nv, tails, lengths)
        attn = xp.make_attn(q, out, 0, prompt_len, width * page, 1 / math.sqrt(D))
        xp.xp_prefix_attention(cache.handle, attn, q, table[0, :prompt_pages], tails, lengths, out, None,
                               cache.attention_workspace(attn))
        logits = target.logits(x, out)
        u = torch.rand(N, B - 1, generator=g).cuda()
        noise = torch.empty(N, V).exponential_(generator=g).clamp_(min=1e-20).cuda()
        xp.xp_verify_drafts(drafter.head.handle, logits, draft, blk, None, heat, u, noise, tokens, counts,
                            None, drafter.verify_ws)
        if scores is not None:
            score = dict(logprob=torch.empty(N, B, device="cuda"), entropy=torch.empty(N, B, device="cuda"),
                         rank=torch.empty(N, B, **int32),
                         top_ids=torch.empty(N, B, top, dtype=torch.int64, device="cuda"),
                         top_logprobs=torch.empty(N, B, top, device="cuda"))
            xp.xp_token_logprobs(drafter.head.handle, logits, tokens, heat, *score.values(),
                                 drafter.head.logprobs_workspace(N * B, top))
            scores.append(dict(score, logits=logits, tokens=tokens.clone(), heat=heat))
        # the anchor and the accepted drafts stay: as many tokens as were emitted
        keep = kept.clone()
        keep[1:] += counts
        xp.xp_cache_resize(cache.handle, table, lens, keep, refs, table, lens, refs)
        assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK
        assert xp.xp_get_error(drafter.head.handle) == xp.XP_OK
        n_out = counts.cpu().tolist()
        for n, row in enumerate(tokens.cpu().tolist()):
            emitted[n] += row[:n_out[n]]
        accepted += sum(n_out) - N
        last = counts.long() - 1
        before = torch.where(last > 0, tokens.gather(1, (last - 1).clamp(min=0)[:, None])[:, 0], anchor)
        anchor = tokens.gather(1, last[:, None])[:, 0]

    # the last request's place goes to a second continuation of the first, then the pool is packed
    gone = lens.clone()
    gone[N] = 0
    xp.xp_cache_resize(cache.handle, table, lens, gone, refs, table, lens, refs)
    xp.xp_cache_fork(cache.handle, table, lens, torch.tensor([1], **int32), None, refs, table[N:],
                     lens[N:], refs)
    live = torch.zeros(1, **int32)
    xp.xp_cache_compact(cache.handle, table, lens, refs, table, refs, None, live)
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK
    held = table[table >= 0]
    assert int(live) == held.unique().numel() and int(held.max()) < int(live)
    return target, prompt, start, emitted, accepted, steps * N * (B - 1)


def main():
    for sampled in (False, True):
        _, _, _, emitted, accepted, made = run(temperature=0.8, dtype=torch.bfloat16, sampled=sampled)
        print("%s drafts accepted: %d of %d" % ("sampled" if sampled else "greedy", accepted, made))
        for n, row in enumerate(emitted):
            print("request %d: %s" % (n, row))
    for bits in (8, 4):
        scores = []
        _, _, _, emitted, accepted, made = run(temperature=0.8, dtype=torch.bfloat16, bits=bits, scores=scores)
        print("a cache of %d bits: accepted %d of %d" % (bits, accepted, made))
        for n in range(len(emitted)):
            print("request %d: %s" % (n, ["%.2f" % x for s in scores for t, x in zip(s["tokens"][n], s["logprob"][n])
                                          if t >= 0]))


if __name__ == "__main__":
    main()
