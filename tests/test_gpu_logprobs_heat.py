"""Log probabilities where logits are very large beside the temperature: differences over t pass fp32.

A log probability below fp32's range is -inf.  Where every id but the best is that far away the rest has no
share: the entropy of n equal best ids is log n, to the 2^-21 of one 2^x, the 2^-23 of a logarithm and the rounding
of n additions at most.  Values that fp32 holds are within 2^-22 of themselves besides (difference, 1/t, product)."""
import math

import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import quant_oracle as Q
from test_gpu_logprobs import call, make_head

pytestmark = pytest.mark.gpu


def agree(rows, tokens, heat, top):
    V = rows.shape[2]
    out = call(make_head(V), rows, tokens, heat, top)
    got = {k: t.cpu().numpy() for k, t in out.items()}
    l, heat = rows.double().cpu().numpy(), heat.double().cpu().numpy()
    for n in range(rows.shape[0]):
        lp, h, rank, ids, tops = Q.logprobs(l[n, 0], int(tokens[n, 0]), heat[n], top)
        assert got["rank"][n, 0] == rank and got["top_ids"][n, 0].tolist() == ids, n
        e = 2.0 ** -20 + (V / 256 + 64) * 2.0 ** -24
        assert abs(got["entropy"][n, 0] - h) <= e * (1 + h), (n, got["entropy"][n, 0], h)
        with np.errstate(over="ignore"):
            for x, w in zip([got["logprob"][n, 0], *got["top_logprobs"][n, 0]], [lp, *tops]):
                if np.isfinite(np.float32(w)):
                    assert abs(x - w) <= e + 2.0 ** -21 * abs(w), (n, x, w)
                else:
                    assert x == -np.inf, (n, x, w)


@pytest.mark.parametrize("V", [9, 3001, 40001])
@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("dtype,size,heat", [
    (torch.bfloat16, 2048.0, 2e-38), (torch.bfloat16, 2000.0, 1.2e-38), (torch.bfloat16, 3e38, 1e-3),
    (torch.bfloat16, 1e30, 1e-30), (torch.float32, 3e37, 1e-30), (torch.float32, 1e9, 1.2e-38),
    (torch.float32, 3e38, 1e-8), (torch.float32, 1e30, 1e-38), (torch.float32, 4096.0, 2e-38)])
def test_entropy_of_logits_that_are_large_beside_the_temperature(dtype, size, heat, top, V):
    at = torch.arange(V, device="cuda")
    rows = torch.stack([
        torch.where(at == V // 2, size, size / 2),                      # one best
        torch.where(at % 4 == 1, size, -size),                          # some equal best
        torch.full((V,), size, device="cuda"),                          # all equal
        torch.full((V,), -size, device="cuda"),
        torch.where(at == V - 1, size, 0.0),                            # the best last
        torch.where(at == 0, size, -math.inf),
        torch.where(at % 3 == 0, size, torch.where(at % 3 == 1, math.nan, size / 4)),
        size * (at + 1) / (2.0 * V),                                    # it rises all the way
    ])[:, None].to(dtype)
    for token in (0, V // 2, V - 1):
        agree(rows, torch.full((8, 1), token, device="cuda"), torch.full((8,), heat, device="cuda"), top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinite_and_lowest_logits_at_small_temperatures(dtype):
    """+inf reads as fp32's largest value, beside which nothing else has a share."""
    V, info = 5003, torch.finfo(dtype)
    rows = torch.zeros(4, 1, V, device="cuda")
    rows[0, 0, [7, 4000]] = math.inf
    rows[1] = info.min
    rows[1, 0, [2, 5002]] = info.max
    rows[2] = info.min
    rows[3, 0, 100:] = info.min
    rows = rows.to(dtype)
    for heat in (1.2e-38, 1e-30, 1e-7, 1.0):
        agree(rows, torch.full((4, 1), 2, device="cuda"), torch.full((4,), heat, device="cuda"), 5)
