"""The hybrid decode example end to end: every call of a decode step in one
model, its steps against its verify, and the rollback of rejected drafts."""

import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from examples.hybrid_decode import HybridModel

pytestmark = pytest.mark.gpu


def test_verify_gives_the_steps_logits_and_commit_follows_them():
    """Four tokens as steps against the same four as one verify: the logits
    agree to bf16's rounding along the layers (each of 4 layers rounds about 6
    times at 2^-8 of its values: 4 x 6 x 2^-8 < 0.1 of the logits' norm), and
    after committing two drafts a step continues where two steps would be."""
    B = 3
    tokens = torch.randint(0, 1000, (B, 20), generator=torch.Generator().manual_seed(0)).cuda()
    a, b = HybridModel(B, 64), HybridModel(B, 64)
    for j in range(12):
        assert torch.equal(a.step(tokens[:, j]), b.step(tokens[:, j]))
    steps = torch.stack([a.step(tokens[:, 12 + j]) for j in range(4)], 1)
    verified = b.verify(tokens[:, 12:16])

    def off(x, y):
        return float((x - y).norm() / y.norm())

    assert off(verified, steps) < 0.1
    b.commit(torch.full((B,), 2, dtype=torch.int32, device="cuda"))
    assert b.pos.tolist() == [14] * B
    c = HybridModel(B, 64)
    for j in range(14):
        c.step(tokens[:, j])
    assert off(b.step(tokens[:, 14]), c.step(tokens[:, 14])) < 0.1
    for m in (a, b, c):
        assert L.lin_state_read_status(m.status) == 0
