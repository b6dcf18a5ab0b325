"""The hybrid decode example's refusals. CPU only."""

import pytest
import torch

from examples import hybrid_decode


def test_a_verify_of_one_draft_is_refused(monkeypatch):
    """It would move the linear layers' states as a step does, and the commit that
    follows would move them again."""
    model = object.__new__(hybrid_decode.HybridModel)
    monkeypatch.setattr(hybrid_decode.HybridModel, "forward", lambda *a, **k: pytest.fail("ran"))
    for n in (0, 1):
        with pytest.raises(ValueError, match="2 drafts or more"):
            model.verify(torch.zeros((3, n), dtype=torch.int64))


def test_no_steps_leave_nothing_to_verify(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["hybrid_decode.py", "--steps", "0"])
    with pytest.raises(SystemExit):
        hybrid_decode.main()
    assert "--steps" in capsys.readouterr().err
