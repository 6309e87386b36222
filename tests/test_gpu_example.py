"""The example's loop of drafting, scoring, verifying and cutting back, against plain decoding."""
import math

import pytest
import torch

from examples import verify_step

pytestmark = pytest.mark.gpu


def plain_decode(target, prompt, first, count):
    """Greedy decoding one token at a time, attention written out over the whole sequence."""
    tokens = prompt.tolist() + [int(first)]
    for _ in range(count):
        x, q, k, v = (t[0] for t in target.qkv(torch.tensor([tokens], device="cuda")))
        k, v = (t.double().repeat_interleave(target.heads // target.kv_heads, 1) for t in (k, v))
        score = torch.einsum("hd,jhd->hj", q[-1].double(), k) / math.sqrt(target.dim)
        out = torch.einsum("hj,jhd->hd", torch.softmax(score, 1), v).to(x.dtype)
        tokens.append(int(target.logits(x[-1:], out[None]).argmax()))
    return tokens[len(prompt) + 1:]


@pytest.mark.parametrize("prompt_len,page", [(75, 16), (128, 20)])
def test_greedy_blocks_equal_plain_decoding(prompt_len, page):
    target, prompt, start, emitted, accepted, made = verify_step.run(prompt_len=prompt_len, page=page)
    assert 0 < accepted < made
    for first, got in zip(start.tolist(), emitted):
        assert got == plain_decode(target, prompt, first, len(got))


def test_sampled_bf16_runs():
    _, _, _, emitted, accepted, made = verify_step.run(temperature=0.8, dtype=torch.bfloat16, requests=3)
    assert all(len(e) >= 6 for e in emitted) and accepted <= made
