"""The training example end to end: the distilled head's loss falls and its expected acceptance
rises, and the answered tokens' log probabilities are the target's."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_training_raises_the_expected_acceptance():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("train_draft_head", os.path.join(ROOT, "examples", "train_draft_head.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history, answer, lp = example.main(steps=150, log=lambda *_: None)
    first, last = history[:10], history[-10:]
    mean = lambda rows, k: sum(r[k] for r in rows) / len(rows)  # noqa: E731
    assert mean(last, 0) < mean(first, 0)
    assert mean(last, 1) > mean(first, 1) + 0.02
    given = answer >= 0
    assert given[:, 0].all()                       # every request answers at least one token
    assert (lp["logprob"][given] < 0).all() and (lp["rank"][given] >= 1).all()
    assert (lp["logprob"][~given] == 0).all() and (lp["top_ids"][~given] == -1).all()
