"""GPU: the example that runs cache, attention, experts and draft verification together.

The greedy run's tokens are looked up in the logits of a second pass over each whole
sequence with a cache of its own.  There the pages' scales can differ from the run's (a
rejected draft may have raised one), so keys and values differ by E4M3 roundings, 2^-4 of
each, which averages to a few percent of a row's attention output and less of its logits:
a token must come within a quarter of the row's standard deviation of the largest logit
(a wrong cache, mask or verdict gives tokens that are several below)."""
import importlib.util
import pathlib

import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "speculative_step.py"
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_greedy_tokens_are_the_models(example):
    prompt = 20
    model, hist, taken = example.generate("greedy", prompt=prompt)
    assert any(n > 0 for step in taken for n in step)  # some drafts are right
    fresh = example.Model(len(hist), max(map(len, hist)) + 32)
    for b, h in enumerate(hist):
        logits = fresh.prompt(b, h).float()
        for t in range(prompt, len(h)):
            row = logits[t - 1]
            assert row[h[t]] >= row.max() - 0.25 * row.std(), (b, t)


@pytest.mark.parametrize("mode", ["sampled", "lookup"])
def test_sampled_runs(example, mode):
    _, hist, taken = example.generate(mode, steps=6)
    assert all(0 <= t < example.VOCAB for h in hist for t in h)
    assert all(len(h) == 20 + sum(step[b] + 1 for step in taken) for b, h in enumerate(hist))
    if mode == "sampled":
        assert any(n > 0 for step in taken for n in step)
    assert example.generate(mode, steps=6)[1] == hist  # bit for bit
