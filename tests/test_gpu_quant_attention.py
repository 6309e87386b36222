"""Attention over caches of 8 and 4 bits against the definition in 64 bits on the values held.

What an output may be off, per row, from the roundings: the output's own (2^-8 of it, half a step of bf16),
the weights' to fp16 (2^-11 of the weighted mean of |v|, A) and the scores': products of fp16 are summed in
fp32 over D dims, each sum within 2^-22 of its terms' size, so a score within dz = (D + 8) 2^-22 scale
sum |q||k|, and a quotient of weighted sums within 2 dz A; sums over n keys within n 2^-23 A; 2^x within
2^-21.  Queries are exact in fp16 where they lie within 2^14 of their row's largest, and lose less than 2^-25 of
that otherwise, which is below dz.  A weight is held as 2^(z - m + 6) with m at most the row's largest
score, so the largest is at least 2^6; where that of a key is below 2^-14, fp16 is a fixed grid of 2^-24 and
it is off by up to 2^-25, 2^-31 of the largest and so of the sum: together 2^-31 sum_j |v_j|.  Codes of 4 bits
are summed as they are held, c + 8 <= 15, and 8 times the weighted mean B of their scales is taken off:
sums of up to 15 B and 8 B, each within (n + 8) 2^-23, (n + 8) 2^-23 23 B together (the least scale that reaches a
group's largest leaves it a code of 3 or more, so a scale is at most a third of what is held there).
lse: dz + n 2^-23 + 2^-21 (1 + |lse|).
Where many queries see each key the cache is widened to fp16 first, exactly, and all else is the same."""
import math

import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import quant_oracle as Q

pytestmark = pytest.mark.gpu


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def build(bits, ps, H, D, prefix, lens, seed, layer=0, layers=1, fill=None):
    """A cache whose first sequence is the prefix; returns it, the tables and the values held."""
    g = np.random.default_rng(seed)
    N = len(lens)
    every = [prefix] + list(lens)
    used = [-(-n // ps) for n in every]
    width, pages = max(1, max(used[1:])), sum(used) + 3
    ids = g.permutation(pages).astype(np.int32)
    k, v = (xp.QuantCache.pool(layers, pages, ps, H, D, bits) for _ in range(2))
    for pool in (k, v):       # a pool is never cleared: scales that are infinities or NaN among what it holds
        pool.copy_(torch.randint(0, 256, pool.shape, device="cuda", dtype=torch.uint8))
    c = xp.QuantCache(k, v, ps, D, bits)
    table, held, at = np.full((N + 1, max(width, used[0], 1)), -1, np.int32), [], 0
    for n, length in enumerate(every):
        table[n, :used[n]] = ids[at:at + used[n]]
        at += used[n]
    T = max(every)
    held = [[np.zeros((n, H, D)) for n in every] for _ in range(2)]
    if T:
        rows = [torch.from_numpy(g.normal(size=(N + 1, T, H, D)).astype(np.float32)).cuda() for _ in range(2)]
        rows[0][:, ::5] *= 3.0
        if fill is not None:
            fill(rows)
        # token t of a row goes to lens - T + t: the rows' last tokens are what is written
        xp.xp_cache_append(c.handle, layer, *rows, cu(table), cu(every))
        assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
        out = [torch.empty(N + 1, T, H, D, device="cuda") for _ in range(2)]
        xp.xp_cache_read(c.handle, layer, cu(table), cu(every), None, *out)
        held = [[o[n, :length].double().cpu().numpy() for n, length in enumerate(every)] for o in out]
    return c, cu(table[0]), cu(table[1:, :width]), held


def check(bits, N, T, H, G, D, ps, prefix, lens, seed=0, layer=0, layers=1, scale=None, q=None, fill=None):
    c, prefix_table, table, held = build(bits, ps, H, D, prefix, lens, seed, layer, layers, fill)
    g = np.random.default_rng(seed + 1)
    scale = scale or 1 / math.sqrt(D)
    if q is None:
        fused = torch.from_numpy(g.normal(size=(N, T, (G + 2) * H, D)) * 1.5).to(torch.bfloat16).cuda()
        q = fused[:, :, :G * H]
    wide = torch.full((N, T, G * H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = wide[:, :, :G * H], torch.full((N, T, G * H), 7.0, device="cuda")
    max_len = max(list(lens) + [0])
    a = xp.make_attn(q, out, layer, prefix, max_len, scale)
    ws = c.attention_workspace(a)
    args = (c.handle, a, q, prefix_table if prefix else None, table if max_len else None,
            cu(lens) if max_len else None)
    xp.xp_prefix_attention(*args, out, lse, ws)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    ws.fill_(0xFF)          # a workspace need not be cleared
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    a2 = xp.make_attn(q, again, layer, prefix, max_len, scale)
    xp.xp_prefix_attention(c.handle, a2, *args[2:], again, lse2, ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)      # and results repeat bit for bit
    assert (wide[:, :, G * H:] == 7.0).all()
    got, got_lse, qs = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for n in range(N):
        k, v = (np.concatenate([h[0], h[n + 1]]) for h in held)
        sees = [prefix + max(0, lens[n] - T + 1 + t) for t in range(T)]
        want, want_lse, mean, size = Q.attention(qs[n], k, v, sees, scale)
        held_as = 0.0
        if bits == 4:
            step = np.abs(v).reshape(len(v), H, D // 16, 16).max(-1).repeat(16, -1) / 3
            held_as = Q.attention(qs[n], k, step, sees, scale)[0] * 23 * (len(k) + 8) * 2.0 ** -23
        dz = (D + 8) * 2.0 ** -22 * size
        tol = 2.0 ** -8 * np.abs(want) + mean * (2.0 ** -11 + 2 * dz + len(k) * 2.0 ** -23 + 2.0 ** -20)[..., None] \
            + 2.0 ** -31 * np.abs(v).sum(0).repeat(G, 0) + held_as + 1e-30
        assert (np.abs(got[n] - want) <= tol).all(), (n, np.max(np.abs(got[n] - want) / tol))
        seen = np.isfinite(want_lse)
        assert (got_lse[n][~seen] == -np.inf).all() and (got[n][~seen] == 0).all()
        tol = dz + len(k) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(seen, want_lse, 0)))
        assert (np.abs(got_lse[n][seen] - want_lse[seen]) <= tol[seen]).all()


CASES = [  # N, T, kv heads, group, dim, page, prefix, lens
    (1, 1, 1, 1, 64, 16, 0, [1]),
    (1, 1, 1, 1, 16, 1, 0, [3]),
    (2, 1, 2, 4, 128, 16, 0, [0, 40]),
    (4, 1, 8, 4, 128, 16, 512, [1, 64, 30, 17]),
    (3, 1, 2, 8, 64, 32, 0, [1000, 129, 127]),
    (3, 1, 1, 7, 128, 8, 33, [500, 0, 1]),
    (7, 5, 3, 4, 96, 20, 1001, [0, 3, 333, 5, 4, 32, 31]),
    (2, 3, 2, 3, 80, 7, 50, [2, 77]),
    (5, 16, 2, 4, 128, 64, 300, [16, 17, 400, 100, 3]),
    (2, 13, 1, 2, 48, 5, 0, [60, 13]),
    (2, 4, 1, 3, 256, 16, 100, [130, 64]),
    (3, 2, 2, 1, 160, 3, 0, [100, 33, 5]),
    (2, 1, 2, 2, 208, 9, 17, [70, 20]),
    (6, 1, 2, 4, 128, 16, 700, [0] * 6),
    (1, 40, 2, 4, 64, 16, 0, [40]),
    (2, 1, 1, 4, 128, 64, 0, [5000, 4000]),
    # work enough for tiles of 16 and of 32 queries
    (64, 4, 4, 4, 128, 16, 0, [130 + i for i in range(64)]),
    (64, 4, 4, 4, 64, 20, 0, [130 + 2 * i for i in range(64)]),
    (64, 3, 4, 3, 256, 16, 0, [130 + i for i in range(64)]),
    (40, 6, 4, 4, 128, 16, 0, [260 + 2 * i for i in range(40)]),
    (40, 6, 4, 4, 96, 7, 0, [260 + 2 * i for i in range(40)]),
    (40, 6, 4, 4, 64, 32, 0, [260 + 2 * i for i in range(40)]),
    (8, 6, 4, 4, 128, 16, 3000, [20 + 9 * i for i in range(8)]),
    # more sequences than a CTA has threads; one that every CTA has a piece of
    (300, 1, 1, 2, 64, 8, 0, [i % 41 for i in range(300)]),
    (1, 1, 1, 4, 64, 64, 0, [30000]),
    (1, 2, 1, 4, 128, 32, 0, [20011]),
    (2, 1, 1, 1, 256, 48, 9001, [0, 700]),
    # many queries a key: the prefix, the tails or both are widened first
    (70, 1, 2, 4, 128, 16, 700, [1 + 5 * i % 90 for i in range(70)]),
    (40, 1, 1, 8, 64, 20, 129, [7 * i % 150 for i in range(40)]),
    (20, 5, 2, 3, 128, 64, 1000, [3 * i for i in range(20)]),
    (33, 1, 3, 8, 128, 8, 128, [0] * 33),
    (3, 40, 2, 4, 64, 16, 0, [300, 40, 7]),
    (2, 150, 2, 2, 128, 20, 130, [150, 400]),
    (5, 16, 1, 4, 128, 64, 40, [0, 16, 128, 129, 500]),
    (1, 300, 1, 1, 64, 16, 5, [300]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("bits", [4, 8])
def test_against_the_definition(case, bits):
    check(bits, *case, seed=sum(case[:7]))


@pytest.mark.parametrize("bits", [4, 8])
def test_widened_layers_and_values_of_any_size(bits):
    def fill(rows):
        rows[0][:, :, 0] *= 1e-4
        rows[1][:, :, 1] *= 8000.0 if bits == 8 else 100.0
        rows[1][:, 3] *= 1e-5
    check(bits, 20, 4, 2, 4, 128, 16, 200, [70 + i for i in range(20)], layer=1, layers=3, fill=fill)
    check(bits, 4, 20, 2, 4, 64, 16, 200, [70 + i for i in range(4)], layer=2, layers=3, fill=fill, scale=0.4)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_layer_of_several_and_another_scale(bits):
    check(bits, 3, 2, 2, 2, 64, 16, 40, [33, 0, 90], layer=2, layers=3, scale=0.7)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size", [1e-30, 1e-4, 3e3, 1e30])
def test_queries_of_any_size(bits, size):
    """Largest, smallest and mixed queries: only their order of magnitude within a row is lost."""
    g = np.random.default_rng(7)
    q = torch.from_numpy(g.normal(size=(2, 2, 4, 128)) * size).to(torch.bfloat16).cuda()
    q[0, 0, 0] = 0
    q[1, 1, 2, ::3] *= 1e-3
    check(bits, 2, 2, 2, 2, 128, 16, 20, [70, 40], q=q, scale=min(1.0, 1 / size) * 0.1)
    check(bits, 2, 70, 2, 2, 128, 16, 20, [170, 40], q=q.repeat(1, 35, 1, 1), scale=min(1.0, 1 / size) * 0.1)


def test_large_and_small_values():
    def fill(rows):
        rows[0][:, :, 0] *= 1e-4
        rows[1][:, :, 1] *= 8000.0
        rows[1][:, 3] *= 1e-5
    check(8, 3, 2, 2, 2, 64, 16, 20, [70, 40, 3], fill=fill)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T", [2, 140])
def test_a_query_that_is_not_finite_spoils_its_row_alone(bits, T):
    c, prefix_table, table, _ = build(bits, 16, 2, 64, 40, [30, 70], 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, T, 4, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    outs = []
    for bad in (None, math.nan, math.inf):
        x = q.clone()
        if bad is not None:
            x[1, T - 2, 2, 5] = bad
        out = torch.empty_like(x)
        a = xp.make_attn(x, out, 0, 40, 70, 0.1)
        xp.xp_prefix_attention(c.handle, a, x, prefix_table, table, cu([30, 70]), out, None,
                               c.attention_workspace(a))
        outs.append(out)
    for out, bad in zip(outs[1:], (math.nan, math.inf)):
        mask = torch.ones(2, T, 4, dtype=torch.bool, device="cuda")
        mask[1, T - 2, 2] = False
        assert torch.equal(out[mask], outs[0][mask])
        assert torch.isnan(out[1, T - 2, 2]).any()


def test_lengths_beyond_the_limit_and_bad_pages_are_told():
    c, prefix_table, table, held = build(4, 16, 1, 64, 0, [64, 64], 4)
    q = torch.randn(2, 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    out = torch.empty_like(q)
    a = xp.make_attn(q, out, 0, 0, 64, 0.1)
    ws = c.attention_workspace(a)
    xp.xp_prefix_attention(c.handle, a, q, None, table, cu([64, 64]), out, None, ws)
    fine = out.clone()
    xp.xp_prefix_attention(c.handle, a, q, None, table, cu([99, 64]), out, None, ws)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_ELENGTH and torch.equal(out, fine)
    xp.xp_prefix_attention(c.handle, a, q, None, table, cu([-5, 64]), out, None, ws)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_ELENGTH
    assert (out[0] == 0).all() and torch.equal(out[1], fine[1])
    table[0, 1] = 10 ** 6
    xp.xp_prefix_attention(c.handle, a, q, None, table, cu([64, 64]), out, None, ws)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_EBADPAGE and torch.equal(out[1], fine[1])


def test_streams_and_graphs_with_a_workspace_each():
    c, prefix_table, table, _ = build(4, 16, 2, 128, 300, [100, 40], 5)
    lens = cu([100, 40])
    outs, graphs, want = [], [], []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(i)
        q = torch.randn(2, 3, 8, 128, generator=g, device="cuda", dtype=torch.bfloat16)
        out = torch.empty_like(q)
        a = xp.make_attn(q, out, 0, 300, 100, 0.09)
        ws = c.attention_workspace(a)
        xp.xp_prefix_attention(c.handle, a, q, prefix_table, table, lens, out, None, ws)
        want.append(out.clone())
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            xp.xp_prefix_attention(c.handle, a, q, prefix_table, table, lens, out, None, ws)
        graphs.append((graph, side, q, ws, a))
        outs.append(out.fill_(0))
    for _ in range(3):
        for graph, side, *_ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("T", [1, 70])
def test_pages_past_two_to_the_31_bytes(T):
    ps, H, D, bits = 64, 2, 128, 4
    size = xp.xp_quant_head_bytes(ps, D, bits)
    pages = 2 ** 31 // (H * size) + 5
    g = np.random.default_rng(8)
    rows = [torch.from_numpy(g.normal(size=(1, 200, H, D)).astype(np.float32)).cuda() for _ in range(2)]
    q = torch.from_numpy(g.normal(size=(1, T, 4, D))).to(torch.bfloat16).cuda()
    outs = []
    for count, ids in ((pages, [pages - 1, pages - 3, 0, pages - 2]), (4, [2, 1, 0, 3])):
        k, v = (xp.QuantCache.pool(1, count, ps, H, D, bits) for _ in range(2))
        c = xp.QuantCache(k, v, ps, D, bits)
        xp.xp_cache_append(c.handle, 0, *rows, cu([ids]), cu([200]))
        out = torch.empty_like(q)
        a = xp.make_attn(q, out, 0, 0, 200, 0.1)
        xp.xp_prefix_attention(c.handle, a, q, None, cu([ids]), cu([200]), out, None, c.attention_workspace(a))
        assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
        outs.append(out)
    assert torch.equal(*outs) and torch.isfinite(outs[0].float()).all()


def test_queries_and_results_off_sixteen_byte_boundaries():
    for T in (1, 80):
        c, prefix_table, table, _ = build(4, 16, 2, 64, 40, [130, 170], 6)
        g = torch.Generator(device="cuda").manual_seed(T)
        q = torch.randn(2, T, 8, 64, generator=g, device="cuda", dtype=torch.bfloat16)
        outs = []
        for shift in (0, 3):
            wide_q = torch.zeros(2, T, 8, 69, device="cuda", dtype=torch.bfloat16)
            wide_o = torch.full_like(wide_q, 7.0)
            x, out = wide_q[..., shift:shift + 64], wide_o[..., shift:shift + 64]
            x.copy_(q)
            a = xp.make_attn(x, out, 0, 40, 170, 0.1)
            xp.xp_prefix_attention(c.handle, a, x, prefix_table, table, cu([130, 170]), out, None,
                                   c.attention_workspace(a))
            assert (wide_o[..., :shift] == 7).all() and (wide_o[..., shift + 64:] == 7).all()
            outs.append(out.clone())
        assert torch.equal(*outs)


def test_refusals():
    c, prefix_table, table, _ = build(4, 16, 1, 64, 20, [64], 4)
    q = torch.randn(1, 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    out, lens = torch.empty_like(q), cu([64])
    a = xp.make_attn(q, out, 0, 20, 64, 0.1)
    ws = c.attention_workspace(a)

    def call(code, cache=c, attn=a, q=q, prefix=prefix_table, table=table, out=out, ws=ws):
        with pytest.raises(xp.XPError) as e:
            xp.xp_prefix_attention(cache.handle, attn, q, prefix, table, lens, out, None, ws)
        assert e.value.code == code

    f = q.float()
    call(xp.XP_EINVAL, attn=xp.make_attn(f, torch.empty_like(f), 0, 20, 64, 0.1), q=f, out=torch.empty_like(f))
    narrow = q[..., :48].contiguous()
    call(xp.XP_EINVAL, attn=xp.make_attn(narrow, torch.empty_like(narrow), 0, 20, 64, 0.1), q=narrow,
         out=torch.empty_like(narrow))
    call(xp.XP_EINVAL, attn=xp.make_attn(q, out, 1, 20, 64, 0.1))
    call(xp.XP_EINVAL, prefix=prefix_table[:1])
    call(xp.XP_EINVAL, table=table[:, :1].contiguous())
    call(xp.XP_ECAPACITY, ws=ws[:256])
    rows = torch.zeros(1, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    for bad in (rows.expand(1, 1, 2, 64), rows[..., :32]):
        with pytest.raises(xp.XPError):
            xp.xp_cache_append(c.handle, 0, bad, bad, table, lens)
        with pytest.raises(xp.XPError):
            xp.xp_cache_read(c.handle, 0, table, lens, None, bad, bad)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
