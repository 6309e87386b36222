"""Verification at small temperatures.

A scaled logit is z = (l - m) / t: the difference, 1 / t and their product are rounded once each, so a
share has relative error (3 |z| + 4) 2^-24, and a row's sum no more than the mean of that over its
shares, below the largest |z| that is kept (90) and the 2^-24 of each of its additions.  prob is held
to 2^-23 (64 + 2 |z_p| + 2 |z_q|) of itself, and a block whose result hangs on less than
2^-23 (64 + 400) is excused."""
import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import step_oracle as S
from test_gpu_verify import Case

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23 * (64 + 400)


def heated(heat, offset, drafts, N=24, B=5, V=700, seed=0, dtype="f32"):
    """Logits offset + t * normal, so that z is spread as usual while l / t is large; drafted ids drawn
    from the drafter, or likely ones."""
    g = np.random.default_rng(seed)
    c = Case(N=N, B=B, V=V, dtype=dtype, drafts=drafts, seed=seed)
    c.temperature = np.full(N, heat, np.float32)
    z = g.normal(size=(N, B, V)) * 2.5
    c.target = torch.from_numpy((offset + heat * z).astype(np.float32)).to(xp.torch_dtype(dtype)).cuda()
    t = c.target[:, :-1].float().cpu().numpy().astype(np.float64)
    if drafts:
        near = z[:, :-1] + g.normal(size=(N, B - 1, V)) * 0.5
        c.draft = (offset + heat * near).astype(np.float32).reshape(N * (B - 1), V)
        t = c.draft.reshape(t.shape).astype(np.float64)
    c.blk[:, 1:] = ((t - t.max(-1, keepdims=True)) / heat - np.log(g.exponential(size=t.shape))).argmax(-1)
    return c


def held(c, tokens=True):
    got = c.run()
    assert c.error == xp.XP_OK
    want = c.want()
    sure = want[3] > 4 * EPS
    assert sure.sum() >= c.N - 1 - c.N // 50
    assert np.array_equal(got[1][sure], want[1][sure])
    if tokens:
        assert np.array_equal(got[0][sure], want[0][sure])
    heat = c.temperature.astype(np.float64)[:, None]

    def depth(rows):      # |z| of the drafted ids
        rows = rows.astype(np.float64)
        at = np.take_along_axis(rows, c.blk[:, 1:, None], 2)[..., 0]
        return (rows.max(-1) - at) / heat

    z = depth(c.target[:, :-1].float().cpu().numpy())
    if c.draft is not None:
        z = z + depth(c.draft.reshape(c.N, c.B - 1, c.V))
    assert np.all(np.abs(got[2] - want[2])[sure] <= (2.0 ** -23 * (64 + 2 * z) * want[2])[sure])


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("heat,offset", [(1e-3, 20.0), (1e-4, -3.0), (1.0, 3e4)])
def test_tests_of_slots_at_large_scaled_logits(heat, offset, drafts):
    held(heated(heat, offset, drafts), tokens=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tests_of_slots_at_tiny_temperatures(dtype):
    # scaled apart, logits 5 and 20 would both be the largest float; below the least normal float
    # a block is greedy
    heats = [2e-38, 1.2e-38, 1e-37, 1e-39, 1e-45, 1e-30, -1e-38]
    c = Case(N=len(heats), B=4, V=300, dtype=dtype, drafts=False, seed=1)
    c.temperature = np.array(heats, np.float32)
    c.target[:] = 5
    c.target[:, :, 100] = 20
    c.blk[:, 1:] = 100
    c.blk[:, 2] = 7               # refused, however large 5 / t is
    c.u[:, 1] = 0.0
    tokens, counts, prob = c.run()
    assert c.error == xp.XP_OK
    assert np.array_equal(counts, np.full(c.N, 2)) and (tokens[:, 0] == 100).all()
    assert np.array_equal(prob, np.tile(np.float32([1, 0, 0]), (c.N, 1)))
    assert np.array_equal(counts, c.want()[1]) and np.array_equal(prob, c.want()[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heat,offset", [(0.01, 8.0), (1.0, 3000.0), (0.7, -7000.0), (0.6, 40.0)])
def test_sums_behind_a_large_maximum(heat, offset, dtype):
    # the maximum's scaled value is large enough for its rounding to show in a sum of its own
    c = heated(heat, offset, False, V=5000, dtype=dtype, seed=3)
    held(c, tokens=False)


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("heat,offset", [(0.01, 8.0), (0.01, 100.0), (1e-3, 20.0), (1e-4, -3.0), (1.0, 3e4)])
def test_draws_at_large_scaled_logits(heat, offset, drafts):
    for seed in range(3):
        held(heated(heat, offset, drafts, N=60, seed=seed))
    c = heated(heat, offset, drafts, N=7, V=9001, dtype="bf16", seed=9)   # steps of z: many equal logits
    held(c)


@pytest.mark.parametrize("heat", [1.2e-38, 1e-36, 1e-30, 1e-10])
def test_draws_at_tiny_temperatures(heat):
    # shares are even among a row's equal maxima, and the race decides: the least noise of them
    c = Case(N=6, B=4, V=500, dtype="f32", drafts=False, seed=2)
    c.temperature = np.full(6, heat, np.float32)
    c.target[:] = 5
    c.target[:, :, 100:110] = 20
    c.blk[:, 1:] = 7
    tokens, counts, _ = c.run()
    assert c.error == xp.XP_OK
    best = 100 + c.noise[:, 100:110].argmin(1)
    assert (counts == 1).all() and np.array_equal(tokens[:, 0], best)
    assert np.array_equal(tokens, c.want()[0])


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("heat,offset", [(1.0, 10.0), (0.01, 100.0), (1e-3, 30.0), (1.0, 3e4)])
def test_draws_between_nearly_equal_ratios(heat, offset, drafts):
    # noise in proportion to the weights: all ratios lie within 2%, the best one 1e-3 above the others.
    # A bound that is not one, or a share rounded at its scaled logit's size, loses it.  Weights below
    # half of p, whose difference magnifies its roundings, stay out of the race.
    N, V = 40, 4000
    c = heated(heat, offset, drafts, N=N, B=2, V=V, seed=4)
    g = np.random.default_rng(5)
    c.u[:] = np.float32(1 - 2 ** -24)
    target = c.target.float().cpu().numpy().astype(np.float64)
    best = np.zeros(N, np.int64)
    for n in range(N):
        p = S.softmax(target[n, 0], heat)
        q = S.softmax(c.draft[n], heat) if drafts else np.zeros(V)
        c.blk[n, 1] = np.argmax(q - p) if drafts else np.argmin(p)       # a draft that is refused
        q = q if drafts else (np.arange(V) == c.blk[n, 1]).astype(float)
        w = np.maximum(p - q, 0)
        best[n] = g.choice(np.nonzero((w > 0.5 * p) & (p > 1e-6))[0])
        spread = g.uniform(0.0, 0.02, V)
        spread[best[n]] = -1e-3
        c.noise[n] = np.where((w > 0.5 * p) & (w > 1e-30), w * np.exp(spread), 1e3).astype(np.float32)
    tokens, counts, _ = c.run()
    assert c.error == xp.XP_OK
    assert (counts == 1).all() and np.array_equal(tokens[:, 0], best)
