"""The quantised cache's calls and the log probabilities together, as a serving loop makes them."""
import math

import numpy as np
import pytest
import torch

from examples import verify_step
from jacobi_speculative_decode_gb300 import xp
from oracle import quant_oracle as Q

pytestmark = pytest.mark.gpu


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads,group,dim,page", [(2, 4, 64, 16), (3, 2, 80, 7)])
def test_blocks_scored_cut_back_forked_and_packed(bits, heads, group, dim, page):
    """Every step: room for a block, its rows in, attention, some tokens cut off again.  What each sequence
    holds is kept as lists of values beside it; the attention's outputs have to follow those (within half a step of
    bf16, 2^-8, and 2^-10 of the weighted mean of |v| for the weights' rounding to fp16 and the scores')."""
    g = np.random.default_rng(bits + dim)
    N, T, layers, prefix = 3, 5, 2, 37
    pages, width = 60, 12
    k, v = (xp.QuantCache.pool(layers, pages, page, heads, dim, bits) for _ in range(2))
    c = xp.QuantCache(k, v, page, dim, bits)
    table, lens, refs = cu(np.full((N + 1, width), -1)), cu(np.zeros(N + 1)), cu(np.zeros(pages))
    held = [[[np.zeros((0, heads, dim)) for _ in range(2)] for _ in range(layers)] for _ in range(N + 1)]

    def write(rows, first, count):
        """`count` new tokens of rows first.. in every layer; their values are kept"""
        for layer in range(layers):
            x = [torch.from_numpy(g.normal(size=(len(rows), count, heads, dim))).to(torch.bfloat16).cuda()
                 for _ in range(2)]
            xp.xp_cache_append(c.handle, layer, *x, table[first:first + len(rows)], lens[first:first + len(rows)])
            for i, n in enumerate(rows):
                for kv in range(2):
                    codes, byte, _ = Q.quantise(x[kv][i].double().cpu().numpy(), bits)
                    held[n][layer][kv] = np.concatenate([held[n][layer][kv], Q.values(codes, byte)])

    def attend(count):
        for layer in range(layers):
            q = torch.from_numpy(g.normal(size=(N, count, heads * group, dim))).to(torch.bfloat16).cuda()
            out = torch.empty_like(q)
            a = xp.make_attn(q, out, layer, prefix, width * page, 1 / math.sqrt(dim))
            xp.xp_prefix_attention(c.handle, a, q, table[0, :-(-prefix // page)], table[1:], lens[1:], out, None,
                                   c.attention_workspace(a))
            for n in range(N):
                kk, vv = (np.concatenate([held[0][layer][kv], held[n + 1][layer][kv]]) for kv in range(2))
                sees = [len(kk) - count + 1 + t for t in range(count)]
                want, _, mean, _ = Q.attention(q[n].double().cpu().numpy(), kk, vv, sees, 1 / math.sqrt(dim))
                assert (np.abs(out[n].double().cpu().numpy() - want) <=
                        2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mean + 1e-6).all()

    xp.xp_cache_resize(c.handle, table, lens, cu([prefix, 0, 0, 0]), refs, table, lens, refs)
    write([0], 0, prefix)
    for step in range(4):
        now = lens.cpu().numpy()
        xp.xp_cache_resize(c.handle, table, lens, cu(now + [0, T, T, T]), refs, table, lens, refs)
        write([1, 2, 3], 1, T)
        attend(T)
        keep = now + np.array([0] + [int(x) for x in g.integers(1, T + 1, N)], np.int32)
        xp.xp_cache_resize(c.handle, table, lens, cu(keep), refs, table, lens, refs)
        for n in range(1, N + 1):
            held[n] = [[x[:keep[n]] for x in kv] for kv in held[n]]
    # the last sequence's place goes to a second continuation of the first, and the pool is packed
    gone = lens.clone()
    gone[N] = 0
    xp.xp_cache_resize(c.handle, table, lens, gone, refs, table, lens, refs)
    xp.xp_cache_fork(c.handle, table, lens, cu([1]), None, refs, table[N:], lens[N:], refs)
    held[N] = [[x.copy() for x in kv] for kv in held[1]]
    live = cu([0])
    xp.xp_cache_compact(c.handle, table, lens, refs, table, refs, None, live)
    assert int(table.max()) < int(live)
    for row, layer in ((1, 0), (N, 1), (0, 1)):
        n = int(lens[row])
        ko, vo = (torch.empty(1, n, heads, dim, device="cuda") for _ in range(2))
        xp.xp_cache_read(c.handle, layer, table[row:row + 1], lens[row:row + 1], None, ko, vo)
        for got, want in zip((ko, vo), held[row][layer]):
            assert (got[0].double().cpu().numpy() == want).all()
    now = lens.cpu().numpy()
    xp.xp_cache_resize(c.handle, table, lens, cu(now + [0, 1, 1, 1]), refs, table, lens, refs)
    write([1, 2, 3], 1, 1)                                    # both continuations go their own ways
    attend(1)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK


@pytest.mark.parametrize("bits", [0, 4, 8])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_the_examples_scores(bits, temperature):
    """The log probabilities that come with the emitted tokens, from the logits they were drawn from.  A sum of
    512 terms within 2^-19, and logits of a few units: 1e-5."""
    scores = []
    _, _, _, emitted, accepted, made = verify_step.run(requests=3, dtype=torch.bfloat16, bits=bits, scores=scores,
                                                       temperature=temperature)
    assert accepted <= made and len(scores) == 6
    seen = [[] for _ in emitted]
    for s in scores:
        p = torch.log_softmax(s["logits"].double() / (temperature or 1.0), -1)
        for n, row in enumerate(s["tokens"].tolist()):
            for b, x in enumerate(row):
                if x < 0:
                    assert s["logprob"][n, b] == 0 and s["rank"][n, b] == 0 and s["top_ids"][n, b, 0] == -1
                    continue
                seen[n].append(x)
                order = torch.sort(s["logits"][n, b].float(), descending=True, stable=True)[1].tolist()
                assert s["rank"][n, b] == order.index(x) + 1 and s["top_ids"][n, b].tolist() == order[:3]
                if temperature:
                    assert abs(s["logprob"][n, b] - p[n, b, x]) < 1e-5
                    assert abs(s["entropy"][n, b] + (p[n, b].exp() * p[n, b]).sum()) < 1e-5
                else:
                    assert s["logprob"][n, b] == 0 and s["rank"][n, b] == 1 and s["entropy"][n, b] == 0
    assert seen == emitted
