"""The hybrid prompt example end to end: a prompt in chunks, whole, and token by token."""

import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from examples.hybrid_decode import VOCAB
from examples.hybrid_prompt import HybridPromptModel, chunks

pytestmark = pytest.mark.gpu


def off(x, y):
    return float((x - y).norm() / y.norm())


def test_chunks_steps_and_whole_prompts_give_the_same_logits():
    """To bf16's rounding along the layers: each of 4 layers rounds about 6 times at 2^-8
    of its values, and its conv's activation is off by up to 2^-11 in a prompt:
    4 x 7 x 2^-8 < 0.11 of the logits' norm."""
    lengths, B = [70, 200, 1], 3
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randint(VOCAB, (n,), generator=gen).cuda() for n in lengths]
    whole, parts, steps = (HybridPromptModel(B, 256) for _ in range(3))
    want = whole.prompt(torch.cat(prompts), lengths).split(lengths)
    got = [[] for _ in lengths]
    for done, new in chunks(lengths, 64):
        out = parts.prompt(torch.cat([p[d:d + n] for p, d, n in zip(prompts, done, new)]), new)
        for r, x in enumerate(out.split(new)):
            got[r].append(x)
    for r in range(B):
        assert off(torch.cat(got[r]), want[r]) < 0.11
    assert parts.pos.tolist() == whole.pos.tolist() == lengths
    # a step after the prompts, against prompts that are one token longer
    token = torch.tensor([5, 6, 7], device="cuda")
    longer = HybridPromptModel(B, 256)
    after = longer.prompt(torch.cat([x for p, t in zip(prompts, token) for x in (p, t[None])]), [n + 1 for n in lengths])
    last = torch.stack([x[-1] for x in after.split([n + 1 for n in lengths])])
    assert off(whole.step(token), last) < 0.11 and off(parts.step(token), last) < 0.11
    # and the first tokens one by one
    for j in range(20):
        x = steps.step(torch.stack([p[min(j, len(p) - 1)] for p in prompts]))
        for r in (0, 1):
            assert off(x[r], want[r][j]) < 0.11
    for m in (whole, parts, steps, longer):
        assert L.lin_state_read_status(m.status) == 0


def test_a_prompt_that_does_not_add_up_is_refused():
    with pytest.raises(ValueError, match="tokens by n_new"):
        HybridPromptModel(2, 64).prompt(torch.zeros(5, dtype=torch.long, device="cuda"), [2, 2])
