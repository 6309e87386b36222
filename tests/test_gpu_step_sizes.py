"""The step's calls at sizes and in company beyond a drafted block's: prompts, and calls at once."""
import math

import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from test_gpu_attention import Case as Attention, reference64
from test_gpu_verify import Case as Verify, make_head

pytestmark = pytest.mark.gpu

PROMPTS = {
    "100 tokens": dict(lens=[100, 37, 230], T=100, H=2, G=4, D=128, P=70, ps=16),
    "333 tokens, heads of 64": dict(lens=[333, 400, 1], T=333, H=3, G=3, D=64, P=0, ps=64),
    "inside a tile": dict(lens=[511, 129, 700], T=511, H=1, G=2, D=128, P=129, ps=24),
    "a whole prompt": dict(lens=[2048, 2500], T=2048, H=2, G=2, D=128, P=0, ps=64),
    "long before it": dict(lens=[5001], T=257, H=1, G=7, D=64, P=333, ps=128),
    "other width": dict(lens=[200, 64], T=130, H=2, G=2, D=80, P=40, ps=20),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(PROMPTS))
def test_attention_over_a_prompt(name, dtype):
    c = Attention(dtype=dtype, seed=len(name), **PROMPTS[name])
    out, lse = c.run()
    assert xp.xp_cache_get_error(c.cache.handle) == xp.XP_OK
    want, want_lse = reference64(c, c.q)
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and not out[empty].any()
    # a score of D fp32 products, |q k| <= sum |q_i k_i|: (D + 4) 2^-24 of that, in a weight twice that
    # and 2^-20; in bf16 a weight's and the output's own rounding
    D, L = c.q.shape[3], c.P + max(c.lens)
    size = c.scale * float(c.q.double().abs().sum(-1).max()) * 5.0
    top = max(np.abs(x).max() for x in [c.vp] + [t[1] for t in c.tails] if x.size)
    dw = 2 * (D + 4) * 2.0 ** -24 * size + 2.0 ** -20
    err = (out.double() - want)[~empty].abs()
    bound = top * (2 * dw + 2 * L * 2.0 ** -24)
    if dtype == "bf16":
        # a weight's rounding, 2^-9 of each, against the largest value; the output's
        bound += top * 2.0 ** -8 + 2.0 ** -8 * want[~empty].abs()
    assert (err <= bound).all()
    assert (lse.double() - want_lse)[~empty].abs().max() <= dw + (L + 20) * 2.0 ** -23
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_verifications_on_two_streams():
    head = make_head(3000, 6, 30, "bf16")
    cases = [Verify(N=30, B=6, V=3000, seed=s, drafts=s == 1) for s in (1, 2)]
    spaces = [head.verify_workspace(30) for _ in cases]
    want = [c.run(head, ws) for c, ws in zip(cases, spaces)]
    cu = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    args = [[c.target, cu(c.draft), cu(c.blk), None, cu(c.temperature), cu(c.u), cu(c.noise)] for c in cases]
    streams, got = [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()
    for _ in range(10):
        for a, ws, s in zip(args, spaces, streams):
            with torch.cuda.stream(s):
                out = [torch.zeros(30, 6, dtype=torch.int64, device="cuda"),
                       torch.zeros(30, dtype=torch.int32, device="cuda"), torch.zeros(30, 5, device="cuda")]
                xp.xp_verify_drafts(head.handle, *a, *out, ws)
                got.append(out)
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for x, y in zip(out, want[i % 2]):
            assert np.array_equal(x.cpu().numpy(), y)
    assert xp.xp_get_error(head.handle) == xp.XP_OK
