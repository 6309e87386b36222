"""Shared-prefix attention against its fp64 statement.

Bounds, from the roundings alone.  A score of fp32 products has error at most
ds = (dim + 4) 2^-24 S, S = scale * max_j sum_i |q_i k_ji|; a weight's relative error is then
dw = 2 ds + 2^-20 (exp2, its argument, rescaling), a sum's a further L 2^-24.  So |d out| <=
max|v| (2 dw + 2 L 2^-24) and |d lse| <= dw + (L + |lse|) 2^-23 for fp32.  In bf16 each weight is rounded once
more (2^-9, independently: held by its root mean square against sqrt(sum p^2 v^2), and elementwise
by max|v| 2^-8), and so is out (2^-9 |out|)."""
import math

import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, T=1, H=2, G=4, D=64, P=0, ps=16, order="token", dtype="bf16", seed=0,
                 sharp=1.5, fused=False, wide=0, layers=1, layer=0, extra_pages=5):
        g = torch.Generator().manual_seed(seed)
        dt = xp.torch_dtype(dtype)
        N = len(lens)
        self.T, self.P, self.lens, self.dtype, self.layer = T, P, lens, dtype, layer
        self.scale = 1 / math.sqrt(D)
        used = [-(-n // ps) for n in lens]
        pp = -(-P // ps)
        pages = pp + sum(used) + extra_pages
        ids = torch.randperm(pages, generator=g).tolist()
        prefix, at, width = ids[:pp], pp, max(1, max(used, default=0)) + wide
        rows = []
        for u in used:
            rows.append(ids[at:at + u] + [-1] * (width - u))
            at += u
        shape = (layers, pages, ps, H, D) if order == "token" else (layers, pages, H, ps, D)
        self.k, self.v = (torch.full(shape, math.nan, dtype=dt, device="cuda") for _ in range(2))
        if order == "head":
            self.k, self.v = self.k.transpose(2, 3), self.v.transpose(2, 3)
        self.tails = []

        def fill(where, count):
            kv = [torch.randn(count, H, D, generator=g).to(dt) for _ in range(2)]
            for i, p in enumerate(where):
                part = slice(i * ps, min(count, (i + 1) * ps))
                self.k[layer, p, :part.stop - part.start] = kv[0][part].cuda()
                self.v[layer, p, :part.stop - part.start] = kv[1][part].cuda()
            return [x.float().numpy() for x in kv]

        self.kp, self.vp = fill(prefix, P)
        for r, n in zip(rows, lens):
            self.tails.append(fill(r[:-(-n // ps)], n))
        q = torch.randn(N, T, H * G + (2 * H if fused else 0), D, generator=g) * sharp
        self.q = q.to(dt).cuda()[:, :, :H * G]
        self.prefix_table = torch.tensor(prefix or [0], dtype=torch.int32, device="cuda")
        self.table = torch.tensor(rows, dtype=torch.int32, device="cuda")
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cache = xp.Cache(self.k, self.v)

    def run(self, max_len=None, out=None, stream=None):
        N, T, heads, D = self.q.shape
        out = torch.full((N, T, heads, D), 7.0, dtype=self.q.dtype, device="cuda") if out is None else out
        lse = torch.full((N, T, heads), 7.0, device="cuda")
        a = xp.make_attn(self.q, out, self.layer, self.P,
                         max(self.lens) if max_len is None else max_len, self.scale)
        ws = self.cache.attention_workspace(a)
        ws.fill_(255)          # what a workspace holds does not matter
        xp.xp_prefix_attention(self.cache.handle, a, self.q, self.prefix_table, self.table,
                               self.lens_t, out, lse, ws, stream)
        return out, lse

    def check(self, got=None):
        out, lse = got or self.run()
        assert xp.xp_cache_get_error(self.cache.handle) == xp.XP_OK
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        wo, wl, spread, size = S.attention(self.q.double().cpu().numpy(), self.kp, self.vp, self.tails,
                                           self.scale)
        empty = np.isneginf(wl)
        assert np.array_equal(empty, np.isneginf(lse)) and not out[empty].any()
        L, D = self.P + max(self.lens), out.shape[-1]
        top = max([np.abs(x).max() for x in [self.vp] + [t[1] for t in self.tails] if x.size] or [0])
        dw = 2 * (D + 4) * 2.0 ** -24 * size + 2.0 ** -20
        assert np.all(np.abs(lse[~empty] - wl[~empty])
                      <= (dw + (L + np.abs(wl)) * 2.0 ** -23)[~empty])
        bound = (top * (2 * dw + 2 * L * 2.0 ** -24))[..., None] + np.zeros_like(out)
        if self.dtype == "bf16":
            rms = lambda x: np.sqrt(np.mean(x * x)) if x.size else 0.0     # noqa: E731
            assert rms(out - wo) <= 2.0 ** -8 * (rms(spread) + rms(wo)) + rms(bound)
            bound = bound + top * 2.0 ** -8 + 2.0 ** -8 * np.abs(wo)
        assert np.all(np.abs(out - wo) <= bound)


CASES = {
    "one key": dict(lens=[1]), "one key wide": dict(lens=[1], D=128, H=1, G=1),
    "prefix only": dict(lens=[0, 0, 0], P=5), "one prefix key": dict(lens=[0], P=1, D=128),
    "nothing": dict(lens=[0, 0], T=2), "some empty": dict(lens=[0, 3, 0, 40, 129], T=4),
    "shorter than the block": dict(lens=[1, 2, 15, 16, 17], T=16, P=33),
    "tile edges": dict(lens=[127, 128, 129, 255, 256, 257], D=128, T=2),
    "prefix tile edges": dict(lens=[5, 0, 9], P=128, T=3, D=128),
    "prefix past an edge": dict(lens=[5, 64, 9], P=257, T=8, D=128, ps=64),
    "long tail": dict(lens=[3000, 7], D=64, G=8, H=1),
    "long prefix": dict(lens=[70, 3, 200], P=5000, T=5, D=128, H=2, G=3),
    "many rows": dict(lens=list(range(0, 120, 3)), P=300, T=16, H=1, G=4, D=128),
    "many rows narrow": dict(lens=[33] * 30, P=700, T=7, H=2, G=5, D=64),
    "heads outside": dict(lens=[100, 31, 64], P=100, T=4, D=128, order="head", ps=32),
    "fused queries": dict(lens=[100, 31, 64], P=100, T=4, D=128, fused=True, ps=128),
    "pages of 24": dict(lens=[100, 24, 25, 23], P=49, T=2, ps=24),
    "pages of 8": dict(lens=[100, 24, 25, 7], P=131, T=2, ps=8, D=128),
    "pages of 256": dict(lens=[300, 24, 511], P=700, T=2, ps=256),
    "pages of 192": dict(lens=[300, 24, 400], P=200, T=2, ps=192),
    "pages of 20": dict(lens=[100, 24, 25, 23], P=49, T=2, ps=20),
    "pages of 1": dict(lens=[10, 3], P=4, T=2, ps=1), "wide table": dict(lens=[40, 3], wide=9),
    "odd width": dict(lens=[70, 5], P=30, T=3, D=40, H=1, G=3), "width 1": dict(lens=[9], D=1),
    "width 80": dict(lens=[70, 130], P=77, T=3, D=80, H=3, G=2), "width 256": dict(lens=[70, 130], P=77, T=3, D=256),
    "width 192": dict(lens=[140], P=7, T=20, D=192, H=1), "layer 2 of 3": dict(lens=[70, 5], P=30, layers=3, layer=2, D=128),
    "sharp": dict(lens=[200, 90], P=300, T=6, D=128, sharp=12.0), "flat": dict(lens=[200, 90], P=300, T=6, sharp=0.01),
    "single heads": dict(lens=[50] * 9, P=200, H=4, G=1, T=1, D=128),
    "big group": dict(lens=[50, 300], P=200, H=1, G=48, T=9, D=64),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_the_statement(name, dtype):
    Case(dtype=dtype, seed=len(name), **CASES[name]).check()


def test_rescaled_maximum():
    # keys whose scores climb from tile to tile, so that every tile raises the running maximum
    c = Case([900], T=3, D=64, H=1, G=2, P=700, seed=3)
    q0 = c.q[0, 0, 0].float()
    for pool, table, count in ((c.k, c.prefix_table, 700), (c.k, c.table[0], 900)):
        for i in range(-(-count // 16)):
            pool[0, table[i]] = (q0 * 0.002 * (i + 1)).to(pool.dtype)
    for kv, table, count in ((c.kp, c.prefix_table, 700), (c.tails[0][0], c.table[0], 900)):
        kv[:] = np.concatenate([c.k[0, p].float().cpu().numpy() for p in table[:-(-count // 16)].tolist()])[:count]
    c.check()


def test_repeats_to_the_bit():
    c = Case([500, 3, 1200, 64], T=16, D=128, H=2, G=4, P=3000, ps=64, seed=9)
    first = c.run()
    for _ in range(5):
        again = c.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_strided_output_and_larger_bound():
    c = Case([90, 3, 33], T=4, D=64, P=40, wide=40, seed=2)
    N, T, heads, D = c.q.shape
    wide = torch.full((N, T, heads + 3, D + 8), 9.0, dtype=c.q.dtype, device="cuda")
    out, lse = c.run(max_len=600, out=wide[:, :, 1:heads + 1, :D])
    c.check((out, lse))
    assert (wide[:, :, 0] == 9).all() and (wide[:, :, :, D:] == 9).all()


@pytest.mark.parametrize("shift", [1, 4])
def test_unaligned_queries(shift):
    # queries and outputs that start between two 16-byte boundaries
    c = Case([90, 200], T=2, D=128, P=40, seed=4)
    flat = torch.empty(c.q.numel() + 8, dtype=c.q.dtype, device="cuda")
    q = flat[shift:shift + c.q.numel()].view(c.q.shape)
    q.copy_(c.q)
    c.q = q
    c.check(c.run(out=torch.empty_like(flat)[shift:shift + q.numel()].view(q.shape)))


def test_no_lse_and_no_tail():
    c = Case([0, 0], T=2, D=128, P=300, seed=5)
    out = torch.empty_like(c.q)
    a = xp.make_attn(c.q, out, 0, c.P, 0, c.scale)
    xp.xp_prefix_attention(c.cache.handle, a, c.q, c.prefix_table, None, None, out, None,
                           c.cache.attention_workspace(a))
    assert torch.equal(out, c.run()[0])


def test_other_stream_and_graph():
    c = Case([90, 200, 5], T=4, D=128, P=500, seed=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
        side.synchronize()
    c.check(got)
    out, lse = torch.empty_like(got[0]), torch.empty_like(got[1])
    a = xp.make_attn(c.q, out, 0, c.P, 200, c.scale)
    ws = c.cache.attention_workspace(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xp.xp_prefix_attention(c.cache.handle, a, c.q, c.prefix_table, c.table, c.lens_t, out, lse, ws)
    c.q.mul_(0.5)            # new values at the captured addresses
    out.fill_(3)
    g.replay()
    c.check((out, lse))


def test_lengths_and_pages_out_of_range():
    c = Case([90, 40], T=2, D=64, P=20, seed=7)
    whole = c.run()[0]
    c.lens_t[0] = 95         # above max_len: read as 90
    out, _ = c.run(max_len=90)
    assert xp.xp_cache_get_error(c.cache.handle) == xp.XP_ELENGTH and torch.equal(out, whole)
    c.lens_t[0] = 90
    c.table[1, 0] = 1 << 20
    c.run()
    assert xp.xp_cache_get_error(c.cache.handle) == xp.XP_EBADPAGE


def test_far_pages():
    # page offsets beyond 2^31 elements
    c = Case([150, 33], T=2, D=128, H=8, G=1, P=200, ps=16, seed=8)
    big = [torch.empty(1, 140000, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pages = c.k.shape[1]
    for b, t in zip(big, (c.k, c.v)):
        b[:, -pages:] = t
    want = c.run()[0]
    c.k, c.v = big
    c.cache = xp.Cache(*big)
    c.prefix_table += 140000 - pages
    c.table[c.table >= 0] += 140000 - pages
    assert torch.equal(c.run()[0], want)
    c.check()


def test_refusals():
    c = Case([90, 40], T=2, D=64, P=20, seed=1)
    out = torch.empty_like(c.q)
    lse = torch.empty(out.shape[:3], device="cuda")

    def code(**kw):
        d = dict(q=c.q, out=out, layer=0, prefix_len=20, max_len=90, scale=0.1, prefix=c.prefix_table,
                 table=c.table, lens=c.lens_t, cut=0, heads=None)
        d.update(kw)
        a = xp.make_attn(d["q"], d["out"], d["layer"], d["prefix_len"], d["max_len"], d["scale"])
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[d["cut"]:]
        if kw.get("small"):
            ws = ws[:256]
        if d["heads"]:
            a.heads = d["heads"]
        try:
            xp.xp_prefix_attention(c.cache.handle, a, d["q"], d["prefix"], d["table"], d["lens"], d["out"],
                                   lse, ws)
        except xp.XPError as e:
            return e.code
        return xp.XP_OK

    assert code() == xp.XP_OK
    assert code(small=True) == xp.XP_ECAPACITY
    for bad in (dict(layer=1), dict(layer=-1), dict(prefix_len=-1), dict(max_len=-1), dict(prefix=None),
                dict(table=None), dict(lens=None), dict(max_len=97), dict(prefix_len=33), dict(cut=8),
                dict(heads=7), dict(q=c.q.float(), out=out.float()), dict(q=c.q[..., :32], out=out[..., :32])):
        assert code(**bad) == xp.XP_EINVAL, bad
    a = xp.make_attn(c.q, out, 0, 20, 90, 0.1)
    with pytest.raises(ValueError):          # not the strides that make_attn was given
        xp.xp_prefix_attention(c.cache.handle, a, c.q.transpose(0, 1), c.prefix_table, c.table, c.lens_t,
                               out, lse, c.cache.attention_workspace(a))
    with pytest.raises(ValueError):
        code(table=c.table.long())
    with pytest.raises(ValueError):
        code(lens=c.lens_t[:1])
    assert xp.xp_cache_get_error(c.cache.handle) == xp.XP_OK


def reference64(c, q):
    """The fp64 definition on the GPU, one sequence at a time (for sizes the CPU statement is slow at)."""
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).double().cuda()     # noqa: E731
    kp, vp = dev(c.kp), dev(c.vp)
    outs, lses = [], []
    for n, length in enumerate(c.lens):
        T, heads, D = q.shape[1:]
        g = heads // kp.shape[1]
        k = torch.cat([kp, dev(c.tails[n][0])]).repeat_interleave(g, 1)
        v = torch.cat([vp, dev(c.tails[n][1])]).repeat_interleave(g, 1)
        score = torch.einsum("thd,jhd->htj", q[n].double(), k) * c.scale
        sees = c.P + (length - T + 1 + torch.arange(T, device="cuda")).clamp(min=0)
        score = score.masked_fill(torch.arange(len(k), device="cuda") >= sees[None, :, None], -math.inf)
        lse = torch.logsumexp(score, -1)
        p = torch.exp(score - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        outs.append(torch.einsum("htj,jhd->thd", p, v))
        lses.append(lse.t())
    return torch.stack(outs), torch.stack(lses)


BATCHES = {
    # shapes whose units are cut between CTAs in different ways: odd row tiles, one tile of a
    # prefix, tails of every length, a row tile pair of one sequence, a long tail alone
    "odd tiles": dict(lens=[(37 * i) % 1500 for i in range(33)], T=5, H=2, G=4, D=128, P=1000, ps=64),
    "single tokens": dict(lens=[(91 * i) % 900 for i in range(150)], T=1, H=4, G=8, D=64, P=3000, ps=32),
    "one row": dict(lens=[(53 * i) % 700 for i in range(90)], T=1, H=8, G=1, D=128, P=129, ps=16),
    "no prefix": dict(lens=[(211 * i) % 2000 for i in range(60)], T=2, H=3, G=3, D=64, P=0, ps=128),
    "wide blocks": dict(lens=[(331 * i) % 600 for i in range(20)], T=16, H=1, G=20, D=128, P=640, ps=64),
    "blocks of 130 rows": dict(lens=[5, 500, 129, 257, 0, 64, 1000], T=13, H=2, G=10, D=64, P=77, ps=24),
    "one long": dict(lens=[0, 20000, 3, 0], T=4, H=2, G=2, D=128, P=20, ps=256),
    "prefix only": dict(lens=[0] * 70, T=3, H=5, G=2, D=128, P=4100, ps=8),
    "tiny tails": dict(lens=[i % 3 for i in range(400)], T=1, H=8, G=4, D=128, P=300, ps=16),
    "pairs of tiles, of heads, and one": dict(lens=[(331 * i) % 900 for i in range(14)], T=16, H=3, G=17,
                                              D=128, P=1000, ps=32),
    "the same narrow": dict(lens=[(57 * i) % 700 for i in range(21)], T=15, H=5, G=18, D=64, P=60, ps=64),
    "odd heads": dict(lens=[(91 * i) % 1300 for i in range(40)], T=2, H=7, G=1, D=128, P=700, ps=16),
    "groups of seven": dict(lens=[(91 * i) % 500 for i in range(50)], T=5, H=4, G=7, D=128, P=333, ps=64),
}


@pytest.mark.parametrize("name", list(BATCHES))
def test_batches_match_the_definition(name):
    c = Case(dtype="bf16", seed=len(name), **BATCHES[name])
    out, lse = c.run()
    assert xp.xp_cache_get_error(c.cache.handle) == xp.XP_OK
    want, want_lse = reference64(c, c.q)
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and not out[empty].any()
    # a weight's and the output's rounding to bf16, 2^-9 each: their root mean square over rows of
    # weights that are spread, three times that for the worst element of |v|max
    err = out.double() - want
    scale = want.square().mean().sqrt() + 1e-3
    assert err.square().mean().sqrt() <= 2.0 ** -8 * 2 * scale
    assert err.abs().max() <= 2.0 ** -8 * (want.abs().max() + 4.5)
    assert (lse.double() - want_lse)[~empty].abs().max() <= 2.0 ** -16
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_calls_on_two_streams():
    cases = [Case([700, 30, 5], T=4, D=128, P=900, seed=s) for s in (11, 12)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(c.run())
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


HIDDEN = {
    "blocks": dict(lens=[1, 2, 7, 129, 300, 131, 0, 16], T=16, H=2, G=4, D=128, P=70, ps=16),
    "cut between ranges": dict(lens=[2900, 40], T=16, H=1, G=2, D=64, P=0, ps=32),
    "row tile pairs": dict(lens=[5, 260, 131, 19], T=20, H=1, G=16, D=128, P=20, ps=64),
    "row tile pairs narrow": dict(lens=[128, 129, 2000], T=13, H=2, G=20, D=64, P=0, ps=24),
    "odd width": dict(lens=[70, 5, 64], P=30, T=6, D=40, H=2, G=3, ps=20),
    "single tokens": dict(lens=[70, 5, 64], P=30, T=1, D=64, H=2, G=3),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(HIDDEN))
def test_what_is_not_finite_reaches_only_the_rows_that_see_it(name, dtype):
    c = Case(dtype=dtype, seed=len(name), **HIDDEN[name])
    out, lse = c.run()
    T, D, ps = c.T, c.q.shape[3], c.k.shape[2]
    heads = c.k.shape[3]
    group = c.q.shape[2] // heads
    odd = [math.inf, math.nan, -math.inf]
    place = lambda n, j: (0, int(c.table[n, j // ps]), j % ps)     # noqa: E731
    sees = lambda n, j: max(0, min(T, j - c.lens[n] + T))          # first row that sees token j  # noqa: E731
    want = out.clone()
    for n, length in enumerate(c.lens):          # values of the last, third last and first tokens
        for i, j in enumerate(sorted({length - 1, length - 3, 0})):
            if 0 <= j < length:
                h, d = (n + i) % heads, (7 * n + 11 * i) % D
                c.v[place(n, j)][h, d] = odd[(n + i) % 3]
                want[n, sees(n, j):, h * group:(h + 1) * group, d] += odd[(n + i) % 3]
    def same(got):
        # a row whose own block held such a value may have been summed in another order, with its
        # weights unrounded: as far off as two roundings of a weight and of the output to bf16
        eps = 2.0 ** -16 if dtype == "f32" else 2.0 ** -7
        for x, y, bound in zip(got, (want, lse), (eps * 5, 2.0 ** -16)):
            assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.isinf(), y.isinf())
            assert torch.equal(x[x.isinf()], y[y.isinf()])
            fine = x.isfinite()
            assert ((x - y)[fine].abs() <= bound).all()

    same(c.run())
    lse = lse.clone()
    for n, length in enumerate(c.lens):          # a key of the last token, of one head
        if length:
            c.k[place(n, length - 1)][n % heads, 3] = math.nan
            rows = (n, slice(sees(n, length - 1), None), slice(n % heads * group, (n % heads + 1) * group))
            want[rows] = math.nan
            lse[rows] = math.nan
    same(c.run())
    assert xp.xp_cache_get_error(c.cache.handle) == xp.XP_OK
