"""Drafts drawn from the refinement's own logits, verified with them."""
import numpy as np
import pytest
import torch

from examples import verify_step
from jacobi_speculative_decode_gb300 import xp
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sampled", [True, False])
def test_first_tokens_follow_the_target(sampled):
    # many requests of the same state: the first token emitted is distributed as the target's softmax,
    # with sampled drafts and their logits as with greedy ones and none
    N, B, V, heat = 4000, 3, 48, 1.6
    target = verify_step.Target(vocab=V, dtype=torch.float32, seed=3)
    drafter = verify_step.Drafter(target, B, N)
    g = torch.Generator().manual_seed(5)
    anchor, before = (torch.full((N,), t, dtype=torch.int64, device="cuda") for t in (7, 11))
    heats = torch.full((N,), heat, device="cuda")
    blk, draft = drafter.sample(anchor, before, heats, g) if sampled \
        else (drafter.draft(anchor, before), None)
    row = torch.randn(B, V, generator=g) * 2
    row[0, target.successor[7].item()] += 4         # near the drafter's own
    logits = row.cuda().expand(N, B, V).contiguous()
    u = torch.rand(N, B - 1, generator=g).cuda()
    noise = torch.empty(N, V).exponential_(generator=g).clamp_(min=1e-20).cuda()
    tokens = torch.empty(N, B, dtype=torch.int64, device="cuda")
    counts = torch.empty(N, dtype=torch.int32, device="cuda")
    prob = torch.empty(N, B - 1, device="cuda")
    xp.xp_verify_drafts(drafter.head.handle, logits, draft, blk, None, heats, u, noise, tokens, counts, prob,
                        drafter.verify_ws)
    assert xp.xp_get_error(drafter.head.handle) == xp.XP_OK
    p = S.softmax(row[0].numpy(), heat)
    assert 0.02 < p[target.successor[7].item()] < 0.9
    seen = np.bincount(tokens[:, 0].cpu().numpy(), minlength=V) / N
    # five standard deviations of a share, and the coarseness of a few
    assert np.all(np.abs(seen - p) < 5 * np.sqrt(p * (1 - p) / N) + 2 / N)
    if sampled:                                     # the drafts follow the logits they came with
        q = S.softmax(draft[0].cpu().numpy(), heat)
        drawn = np.bincount(blk[:, 1].cpu().numpy(), minlength=V) / N
        assert np.all(np.abs(drawn - q) < 5 * np.sqrt(q * (1 - q) / N) + 2 / N)
        want = S.verify(logits[:200].cpu().numpy(), draft[:200 * (B - 1)].cpu().numpy(),
                        blk[:200].cpu().numpy(), None, heats[:200].cpu().numpy(), u[:200].cpu().numpy(),
                        noise[:200].cpu().numpy())
        sure = want[3] > 4 * 2.0 ** -23 * (64 + 400)
        assert sure.sum() >= 195
        assert np.array_equal(tokens[:200].cpu().numpy()[sure], want[0][sure])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_loop_runs_with_sampled_drafts(dtype):
    _, _, _, emitted, accepted, made = verify_step.run(temperature=0.7, dtype=dtype, sampled=True)
    assert all(len(e) >= 6 for e in emitted) and 0 < accepted < made


def test_sampled_drafts_at_temperature_zero_are_greedy():
    plain, drawn = (verify_step.run(temperature=0.0, sampled=s) for s in (False, True))
    assert plain[3] == drawn[3]
