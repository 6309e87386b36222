"""Log probabilities, entropy, rank and alternatives against the definition in 64 bits.

Whole numbers are equal.  The sum S of V terms 2^x is made of at most V/256 + 64 additions in a row, each
within 2^-24, of terms within 2^-21 and 2^-23 |x|, |x| weighted by the terms: its log within
e = 2^-21 + (V/256 + 64) 2^-24 + 2^-22 mean|x|.  A log probability is (l - m)/t - log S: within e plus 2^-22 of
both; the entropy log S - E[x] within e (1 + mean|x|) plus 2^-22 of both."""
import math

import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import quant_oracle as Q

pytestmark = pytest.mark.gpu


def make_head(V, dtype="bf16"):
    r, B = 8, 2
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    shapes = dict(w1=(V, r), down_h=(r, r), down_g=(r, r), in_proj=(r, 3 * r), mix_L=(r, B, B),
                  w_gate=(r, r), w_up=(r, r), w_down=(r, r), w2=(V, r))
    w = {k: torch.zeros(s, dtype=dt, device="cuda") for k, s in shapes.items()}
    return xp.Head(dict(V=V, hidden=r, r=r, H=r, B=B), w, dtype, 4)


def call(head, logits, tokens, temperature, top, ws=None):
    N, B, _ = logits.shape
    f = dict(device="cuda")
    out = dict(logprob=torch.full((N, B), 7.0, **f), entropy=torch.full((N, B), 7.0, **f),
               rank=torch.full((N, B), 7, dtype=torch.int32, **f),
               top_ids=torch.full((N, B, top), 7, dtype=torch.int64, **f),
               top_logprobs=torch.full((N, B, top), 7.0, **f))
    ws = head.logprobs_workspace(N * B, top) if ws is None else ws
    xp.xp_token_logprobs(head.handle, logits, tokens, temperature, *out.values(), ws)
    return out


def check(head, logits, tokens, temperature, top, error=xp.XP_OK, ws=None):
    out = call(head, logits, tokens, temperature, top, ws)
    assert xp.xp_get_error(head.handle) == error
    again = call(head, logits, tokens, temperature, top, ws)
    assert all(torch.equal(out[k], again[k]) for k in out)
    xp.xp_get_error(head.handle)
    got = {k: t.cpu().numpy() for k, t in out.items()}
    rows, toks = logits.double().cpu().numpy(), tokens.cpu().numpy()
    heat = [1.0] * len(rows) if temperature is None else temperature.cpu().double().tolist()
    V = rows.shape[2]
    for n in range(rows.shape[0]):
        for b in range(rows.shape[1]):
            lp, h, rank, ids, tops = Q.logprobs(rows[n, b], toks[n, b], heat[n], top)
            at = (n, b)
            assert got["rank"][at] == rank and got["top_ids"][at].tolist() == ids, at
            l = np.where(np.isnan(rows[at]), -np.inf, np.minimum(rows[at], np.finfo(np.float32).max))
            z, mean = np.zeros(V), 0.0
            if l.max() > -np.inf and heat[n] >= 1.2e-38:
                z = (l - l.max()) / heat[n]
                p = np.exp(z)
                mean = -(p * np.where(p > 0, z, 0.0)).sum() / p.sum()
            e = 2.0 ** -21 + (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -22 * mean * math.log2(math.e)
            log_s = math.log(np.exp(z).sum())

            def near(x, want):
                if not np.isfinite(want):
                    return x == want
                return abs(x - want) <= e + 2.0 ** -22 * (abs(want) + 2 * log_s)
            assert near(got["logprob"][at], lp), (at, got["logprob"][at], lp)
            assert abs(got["entropy"][at] - h) <= (1 + mean) * e + 2.0 ** -22 * (log_s + mean + abs(h)), at
            assert all(near(x, w) for x, w in zip(got["top_logprobs"][at], tops)), at


SIZES = [(1, 1, 5), (1, 8, 151936), (3, 2, 33), (2, 3, 1000), (1, 1, 20011), (40, 16, 4097), (2, 1, 151647)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_against_the_definition(size, dtype, top):
    N, B, V = size
    g = torch.Generator(device="cuda").manual_seed(V + top)
    logits = (torch.randn(N, B, V, generator=g, device="cuda") * 3).to(dtype)
    logits[:, :, V - V // 50:] = -math.inf
    tokens = torch.randint(0, V, (N, B), generator=g, device="cuda")
    tokens[:, ::3] = logits[:, ::3].float().argmax(-1)
    if N * B > 1:
        tokens[0, 0] = -1
    heat = torch.empty(N, device="cuda").uniform_(0.3, 1.7, generator=g)
    heat[N // 2] = 0.0 if N > 2 else 1.0
    check(make_head(V), logits, tokens, None if top == 1 else heat, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", range(1, 8, 3))
def test_rows_off_sixteen_byte_boundaries(dtype, shift):
    V = 2111
    g = torch.Generator(device="cuda").manual_seed(shift)
    wide = torch.randn(3, 4, V + 9, generator=g, device="cuda").to(dtype)
    logits = wide[:, 1:, shift:shift + V]
    check(make_head(V), logits, torch.randint(0, V, (3, 3), generator=g, device="cuda"), None, 7)


def test_ties_and_values_that_are_not_finite():
    V = 5000
    head = make_head(V)
    rows = torch.zeros(8, 1, V, device="cuda")
    rows[1] = torch.arange(V, device="cuda") % 3
    rows[2, 0, :] = -math.inf
    rows[2, 0, [7, 4000]] = 1.5
    rows[3, 0, ::2] = math.nan
    rows[4, 0, [9, 4999]] = math.inf
    rows[5, 0] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)
    rows[6] = torch.linspace(0, 30, V, device="cuda")
    rows[7] = torch.linspace(30, 0, V, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        for token in (0, 1, 7, 9, 2500, 4999):
            check(head, rows.to(dtype), torch.full((8, 1), token, device="cuda"), None, 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1700, 1830, 2049, 9001, 70001, 300007])
def test_rows_that_rise_fall_and_stay(dtype, V):
    """Rows whose best come last, first, or all alike; masked ones with few ids left, and none in some warps."""
    at = torch.arange(V, device="cuda")
    rows = torch.stack([at * (20.0 / V), -at * (20.0 / V), torch.full((V,), 3.0, device="cuda"),
                        torch.where(at % 97 == 5, at % 7 * 1.0, -math.inf),
                        torch.where(at >= V - 3, 1.0, -math.inf), torch.where(at < 40, at * 0.5, -math.inf),
                        torch.full((V,), torch.finfo(dtype).min, device="cuda"),
                        torch.where(at % 256 < 8, -math.inf, (at // 2048 % 5) * 1.0)])[:, None].to(dtype)
    assert torch.isfinite(rows[6].float()).all()
    for top in (32, 3):
        check(make_head(V), rows, torch.full((8, 1), V // 3, device="cuda"), None, top)


def test_large_logits_and_small_temperatures():
    V = 3001
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.randn(4, 1, V, generator=g, device="cuda") * 1e-3
    rows[1] = rows[1] * 1e6 + 1e6
    rows[2] = torch.randn(1, V, generator=g, device="cuda") * 3e37
    rows[3] -= 3e38
    heat = torch.tensor([1e-6, 1e4, 1e37, 1.0], device="cuda")
    check(make_head(V), rows, torch.full((4, 1), 1234, device="cuda"), heat, 4)
    heat = torch.tensor([1e-38, 1e-30, 0.0, -1.0], device="cuda")
    out = call(make_head(V), rows, rows.argmax(-1), heat, 2)
    assert (out["logprob"] <= 0).all() and torch.isfinite(out["logprob"]).all()
    assert (out["logprob"][2:] == 0).all() and (out["entropy"][2:] == 0).all()


def test_empty_rows_and_bad_tokens_are_told():
    V = 700
    head = make_head(V)
    rows = torch.randn(2, 2, V, device="cuda")
    rows[0, 1] = -math.inf
    rows[1, 0] = math.nan
    tokens = torch.tensor([[3, 5], [0, V - 1]], device="cuda")
    check(head, rows, tokens, None, 3, error=xp.XP_EEMPTY)
    for bad in (V, -2, 2 ** 40):
        out = call(head, rows, torch.tensor([[3, bad], [-1, V - 1]], device="cuda"), None, 3)
        assert xp.xp_get_error(head.handle) == xp.XP_EBADTOKEN
        assert out["logprob"][0, 1] == 0 and out["rank"][0, 1] == 0 and (out["top_ids"][0, 1] == -1).all()
        assert out["rank"][0, 0] > 0 and out["rank"][1, 1] > 0


def test_outputs_left_out_and_empty_batches():
    V = 9000
    head = make_head(V)
    rows = torch.randn(2, 3, V, device="cuda", dtype=torch.bfloat16)
    tokens = torch.randint(0, V, (2, 3), device="cuda")
    full = call(head, rows, tokens, None, 4)
    ws = head.logprobs_workspace(6, 4)
    for keep in full:
        out = {k: torch.empty_like(t) if k == keep else None for k, t in full.items()}
        xp.xp_token_logprobs(head.handle, rows, tokens, None, *out.values(), ws)
        assert torch.equal(out[keep], full[keep])
    xp.xp_token_logprobs(head.handle, rows[:0], tokens[:0], None, None, None, None, None, None, ws)
    xp.xp_token_logprobs(head.handle, rows[:, :0], tokens[:, :0], None, None, None, None, None, None, ws)


def test_one_workspace_for_calls_of_any_size():
    """Rows cut and not cut, in turn: the workspace's counts are found at zero by each."""
    V = 40000
    head = make_head(V)
    ws = head.logprobs_workspace(1, 32)
    g = torch.Generator(device="cuda").manual_seed(2)
    for rows, top in ((700, 3), (1, 32), (64, 0), (700, 0), (5, 7), (1, 32)):
        logits = torch.randn(rows, 1, V, generator=g, device="cuda", dtype=torch.bfloat16)
        tokens = torch.randint(0, V, (rows, 1), generator=g, device="cuda")
        out = call(head, logits, tokens, None, top, ws)
        want = torch.log_softmax(logits.double(), -1).gather(2, tokens[:, :, None])[:, :, 0]
        assert (out["logprob"] - want).abs().max() < 1e-4      # a mix-up of rows, not digits
        if top:
            assert torch.equal(out["top_ids"][:, :, 0], logits.float().argmax(-1))


def test_a_stream_and_a_graph():
    V = 151936
    head = make_head(V)
    rows = torch.randn(1, 3, V, device="cuda", dtype=torch.bfloat16)
    tokens = torch.randint(0, V, (1, 3), device="cuda")
    ws = head.logprobs_workspace(3, 5)
    f = dict(device="cuda")
    out = [torch.empty(1, 3, **f), torch.empty(1, 3, **f), torch.empty(1, 3, dtype=torch.int32, **f),
           torch.empty(1, 3, 5, dtype=torch.int64, **f), torch.empty(1, 3, 5, **f)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        xp.xp_token_logprobs(head.handle, rows, tokens, None, *out, ws)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows.copy_(torch.randn(rows.shape, generator=g, **f))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = call(head, rows, tokens, None, 5)
        assert all(torch.equal(a, b) for a, b in zip(out, want.values()))


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinity_beside_the_largest_finite_value(dtype, shift):
    """+inf reads as fp32's largest value: in fp32 rows the two are a tie, whichever comes first."""
    V = 4100
    wide = torch.zeros(4, 1, V + 3, device="cuda", dtype=dtype)
    rows, most = wide[:, :, shift:shift + V], torch.finfo(dtype).max
    rows[0, 0, [1, 40, 2050, 4099]] = torch.tensor([most, math.inf, most, math.inf], device="cuda", dtype=dtype)
    rows[1, 0, [0, 41, 2051, 4098]] = torch.tensor([math.inf, most, math.inf, most], device="cuda", dtype=dtype)
    rows[2, 0, 2048:2056] = torch.tensor([most, math.inf] * 4, device="cuda", dtype=dtype)
    rows[3, 0, 2048:2056] = torch.tensor([math.inf, most] * 4, device="cuda", dtype=dtype)
    for token in (0, 1, 40, 41, 2050, 2051, 2053, 2054, 4098, 4099):
        check(make_head(V), rows, torch.full((4, 1), token, device="cuda"), None, 9)


@pytest.mark.parametrize("size", [(300, 1, 700), (75, 8, 700), (76, 8, 33), (3, 50, 20011), (1, 2, 40000)], ids=str)
def test_rows_without_a_token_among_others(size):
    """Up to as many rows as run at once, cut and whole: half of them without a token."""
    N, B, V = size
    g = torch.Generator(device="cuda").manual_seed(N)
    logits = torch.randn(N, B, V, generator=g, device="cuda", dtype=torch.bfloat16)
    tokens = torch.randint(0, V, (N, B), generator=g, device="cuda")
    tokens[torch.rand(N, B, generator=g, device="cuda") < 0.5] = -1
    tokens[-1, -1] = V - 1
    check(make_head(V), logits, tokens, None, 3)
    check(make_head(V), logits, torch.full_like(tokens, -1), None, 3)


@pytest.mark.parametrize("rise", [-1, 0, 1])
def test_more_batches_than_places(rise):
    """Whole rows of 300000: 74 batches a thread, of which the greatest of 64 are held."""
    V, N = 300000, 620
    g = torch.Generator(device="cuda").manual_seed(5)
    row = torch.randn(1, 1, V, generator=g, device="cuda") + rise * torch.linspace(0, 40, V, device="cuda")
    logits, tokens = row.expand(N, 1, V), torch.full((N, 1), -1, device="cuda")
    at = {3: 0, 300: V - 1, 619: int(row.argmax())}
    for n, token in at.items():
        tokens[n] = token
    out = call(make_head(V), logits, tokens, None, 32)
    got = {k: t.cpu().numpy() for k, t in out.items()}
    for n, token in at.items():
        lp, h, rank, ids, tops = Q.logprobs(row[0, 0].double().cpu().numpy(), token, 1.0, 32)
        assert got["rank"][n, 0] == rank and got["top_ids"][n, 0].tolist() == ids
        # V/256 + 64 additions of 2^-24, and 2^-22 of x below 2^6 and of the differences' mean
        assert abs(got["logprob"][n, 0] - lp) <= 1300 * 2.0 ** -24 + 2.0 ** -15
        assert np.abs(got["top_logprobs"][n, 0] - np.array(tops)).max() <= 1300 * 2.0 ** -24 + 2.0 ** -15
    assert (got["rank"][[0, 2, 618]] == 0).all()
