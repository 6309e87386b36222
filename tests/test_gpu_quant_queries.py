"""Queries of every size over caches of 8 and 4 bits, both forms: what is scaled away for the products is
put back into the scores.

Where scores are of order 1 the tolerances are those of the attention's other tests, which a wrong power of two in a
small query passes by hundreds.  Where one dim of a query holds its only element and the products are huge, a key's score
is one product, exact but for the factor's roundings, which are the same for all keys: the keys with the greatest
share the row equally and no other has a share.  There an output is within 2^-8 of itself (its rounding to bf16)
and 2^-19 of the mean of |v| (n additions of weights that are equal powers of two, n below 2^3); codes of 4 bits add
what the other tests derive for them; lse is the greatest score within 2^-21 (its factor's three roundings, its
own and log 2's)."""
import math

import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from test_gpu_quant_attention import build, check, cu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size", [3e-39, 1e-37, 1e-36, 1e-30, 1e-4, 3e3, 1e30, 1e37])
def test_scores_of_order_one(bits, size):
    g = np.random.default_rng(7)
    q = torch.from_numpy(g.normal(size=(2, 2, 4, 128)) * size).to(torch.bfloat16).cuda()
    q[0, 0, 0] = 0
    q[1, 1, 2, ::3] *= 1e-2
    for T, D in ((2, 128), (70, 128), (2, 96), (70, 64)):
        x = q.repeat(1, T // 2, 1, 1)[..., :D]
        check(bits, 2, T, 2, 2, D, 16, 20, [170, 40], q=x, scale=min(0.1 / size, 3e38))


def huge(bits, size, scale, T, D, lens=(130, 37), G=2, prefix=20):
    H, N = 2, len(lens)

    def fill(rows):   # scores below half of what fp32 holds
        rows[0].mul_(0.05)
    c, prefix_table, table, held = build(bits, 16, H, D, prefix, lens, T + D, fill=fill)
    g = np.random.default_rng(T)
    q = torch.zeros(N, T, H * G, D)
    dims = g.integers(0, D, (N, T, H * G))
    for at in np.ndindex(dims.shape):
        q[at][dims[at]] = size * (1 if g.random() < 0.5 else -1)
    q = q.to(torch.bfloat16).cuda()
    out, lse = torch.empty_like(q), torch.empty(N, T, H * G, device="cuda")
    a = xp.make_attn(q, out, 0, prefix, max(lens), scale)
    xp.xp_prefix_attention(c.handle, a, q, prefix_table, table, cu(lens), out, lse, c.attention_workspace(a))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    got, got_lse, qs = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for n, t, h in np.ndindex(dims.shape):
        k, v = (np.concatenate([x[0], x[n + 1]])[:, h // G] for x in held)
        sees = prefix + max(0, lens[n] - T + 1 + t)
        if sees == 0:
            assert (got[n, t, h] == 0).all() and got_lse[n, t, h] == -np.inf
            continue
        z, v = k[:sees] @ qs[n, t, h] * scale, v[:sees]
        best = v[z == z.max()]
        assert len(best) < 8 and z.max() < 3e38
        want, mean = best.mean(0), np.abs(best).mean(0)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * mean
        if bits == 4:
            step = np.abs(best).reshape(-1, D // 16, 16).max((0, 2)).repeat(16) / 3
            tol = tol + step * 23 * (sees + 8) * 2.0 ** -23
        at = (n, t, h)
        assert (np.abs(got[at] - want) <= tol + 1e-30).all(), (at, got[at], want)
        top = z.max() + math.log(len(best))
        assert abs(got_lse[at] - top) <= 2.0 ** -21 * abs(top) + 2.0 ** -19, (at, got_lse[at], top)


HUGE = [(5e37, 1.0), (1.6e38, 1.0), (1e38, 0.25), (3.0, 2e37), (1e10, 1e28), (6e37, 2.0)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size,scale", HUGE)
@pytest.mark.parametrize("T,D", [(1, 128), (2, 64), (5, 96), (3, 256)])
def test_products_that_are_huge(bits, size, scale, T, D):
    huge(bits, size, scale, T, D)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size,scale", HUGE + [(1e9, 1.0), (1e11, 0.7), (3e7, 3.0)])
@pytest.mark.parametrize("T,D,lens,G,prefix", [
    (70, 64, (130, 37), 2, 20), (70, 128, (130, 37), 2, 0),             # all of it widened
    (70, 128, (1, 3), 2, 0),                                            # one key: a score may be far below 0
    (1, 128, tuple(1 + 3 * i % 200 for i in range(70)), 4, 130),        # the prefix alone
    (3, 64, (300, 0, 2) * 15, 2, 700)], ids=lambda x: str(x)[:16])      # tails beside it
def test_products_that_are_huge_over_widened_keys(bits, size, scale, T, D, lens, G, prefix):
    huge(bits, size, scale, T, D, lens, G, prefix)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,lens,prefix", [(70, (130, 37), 20), (1, tuple(range(1, 200, 2)), 130)],
                         ids=lambda x: str(x)[:16])
@pytest.mark.parametrize("size", [1e6, 1e9, 1e20, 3e37])
def test_a_large_query_beside_others(bits, T, lens, prefix, size):
    """Rows of one tile have nothing to do with one another, and queries turned round get the least score's key."""
    H, G, D, N = 2, 4, 128, len(lens)
    c, prefix_table, table, held = build(bits, 16, H, D, prefix, lens, 3)
    q = torch.randn(N, T, H * G, D, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    at = (N - 1, T // 2, 5)
    outs = []
    for sign in (0, 1, -1):
        x = q.clone()
        if sign:
            x[at] = 0
            x[at][17] = sign * size
        out = torch.empty_like(x)
        a = xp.make_attn(x, out, 0, prefix, max(lens), 0.1)
        xp.xp_prefix_attention(c.handle, a, x, prefix_table, table, cu(lens), out, None, c.attention_workspace(a))
        outs.append(out)
    k, v = (np.concatenate([h[0], h[N]])[:, at[2] // G] for h in held)
    sees = prefix + max(0, lens[-1] - T + 1 + at[1])
    for out, sign in zip(outs[1:], (1, -1)):
        z = sign * k[:sees, 17]
        best = v[:sees][z == z.max()]
        want, got = best.mean(0), out[at].double().cpu().numpy()
        near = 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * np.abs(best).max()
        assert len(best) < 8 and (np.abs(got - want) <= near).all()
        out[at] = outs[0][at]
        assert torch.equal(out, outs[0])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size", [1e5, 3e5, 1e6, 3e6])
@pytest.mark.parametrize("T,lens,prefix", [(2, (130, 37), 20), (70, (130, 37), 20), (1, tuple(range(1, 200, 2)), 5000),
                                           (16, (300, 16, 700), 3000)], ids=lambda x: str(x)[:16])
def test_scores_on_both_sides_of_what_is_summed_again(bits, size, T, lens, prefix):
    """A row's score is one product, exact, and rounded where it is multiplied by its factor, where the maximum is
    and where pieces are joined, within 2^-24 each: dz = 2^-22 of it together, and a weighted mean within 2 dz of
    that of |v|."""
    H, G, D, N = 2, 4, 128, len(lens)

    def fill(rows):
        rows[0].mul_(0.05)
    c, prefix_table, table, held = build(bits, 16, H, D, prefix, lens, 9, fill=fill)
    g = np.random.default_rng(T)
    q = torch.zeros(N, T, H * G, D)
    dims = g.integers(0, D, (N, T, H * G))
    for at in np.ndindex(dims.shape):
        q[at][dims[at]] = size * g.uniform(0.5, 1.0) * (1 if g.random() < 0.5 else -1)
    q = q.to(torch.bfloat16).cuda()
    out, lse = torch.empty_like(q), torch.empty(N, T, H * G, device="cuda")
    a = xp.make_attn(q, out, 0, prefix, max(lens), 1.0)
    xp.xp_prefix_attention(c.handle, a, q, prefix_table, table, cu(lens), out, lse, c.attention_workspace(a))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    got, got_lse, qs = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for n, t, h in np.ndindex(dims.shape):
        k, v = (np.concatenate([x[0], x[n + 1]])[:, h // G] for x in held)
        sees = prefix + max(0, lens[n] - T + 1 + t)
        z, v = k[:sees] @ qs[n, t, h], v[:sees]
        p = np.exp(z - z.max())
        dz = 2.0 ** -22 * np.abs(z[p > 1e-8]).max()
        want, mean = p @ v / p.sum(), p @ np.abs(v) / p.sum()
        # fp16 weights: 2^-11 of each; codes of 4 bits: as in the attention's other tests, a scale is at most |v| / 3
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * dz) * mean + 2.0 ** -31 * np.abs(v).sum(0)
        step = p @ np.abs(v).reshape(sees, D // 16, 16).max(2).repeat(16, 1) / p.sum() / 3
        tol = tol + step * 23 * (sees + 8) * 2.0 ** -23
        assert (np.abs(got[n, t, h] - want) <= tol).all(), (n, t, h)
        top = z.max() + math.log(p.sum())
        assert abs(got_lse[n, t, h] - top) <= 2 * dz + 2.0 ** -22 * abs(top) + 2.0 ** -18, (n, t, h)
