"""GPU: the example that runs pages from lengths, append, attention with shared prefixes, experts and
sampling together.

At temperature 0 each token must come within a quarter of the row's standard deviation of the largest logit
of a second pass over the whole sequence, alone in a cache of its own (pages' scales differ there by what was
appended together, so keys and values by E4M3 roundings; a wrong page, prefix or mask gives tokens that are
several standard deviations below)."""
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
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "parallel_sampling.py"
    spec = importlib.util.spec_from_file_location("parallel_sampling", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_first_tokens_are_the_models(example):
    prompts, samples = (37, 20), 3
    model, hist = example.generate(temperature=0.0, samples=samples, prompts=prompts, steps=10, stop=0.0)
    fresh = example.base.Model(len(hist), max(map(len, hist)) + 32)
    for b, h in enumerate(hist):
        n = prompts[b // samples]
        assert len(h) == n + 10
        logits = fresh.prompt(b, h).float()
        for t in range(n, len(h)):
            row = logits[t - 1]
            assert row[h[t]] >= row.max() - 0.25 * row.std(), (b, t)


def test_pages_are_held_by_those_that_run(example):
    model, hist = example.generate(samples=4, steps=40, stop=0.08)
    refs, table, lens = model.refs.tolist(), model.table.tolist(), model.lens.tolist()
    held = [0] * len(refs)
    for row, n in zip(table, lens):
        for col, page in enumerate(row):
            if col < -(-n // example.PAGE):
                held[page] += 1
            else:
                assert page == -1
    assert refs == held
    assert any(n == 0 for n in lens)  # some have ended
    assert len({tuple(h) for h in hist}) > len(hist) // 2  # samples differ
    assert example.generate(samples=4, steps=40, stop=0.08)[1] == hist  # bit for bit


def test_samples_that_all_end_leave_the_pool_empty(example):
    model, hist = example.generate(samples=2, steps=3, stop=1.0)
    assert int(model.refs.abs().sum()) == 0 and (model.table == -1).all()
    assert all(len(h) == n + 1 for h, n in zip(hist, (37, 37, 20, 20)))
