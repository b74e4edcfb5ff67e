"""The example model end to end: embedding, router, layer, distillation loss
and their gradients train it; the few-token layer answers as the training
path does."""

import importlib.util
import os

import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("small_model", os.path.join(ROOT, "examples", "small_model.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_small_model_trains_and_answers(example):
    model, top_ids, losses = example.train(200)
    assert losses[-1] < 0.2 * losses[0], (losses[0], losses[-1])
    # every token's answer, a few at a time, against the training path's logits
    ids = torch.randperm(example.VOCAB, generator=torch.Generator().manual_seed(3)).int().cuda()
    answers = example.Answers(model, 96)
    few = torch.cat([answers.logits(part) for part in ids.split(96)])
    answers.decoder.check()
    full = model.forward(torch.cat([ids, ids]))[-1][:example.VOCAB]
    # both round a hidden state to bf16 (2^-9 of it) in different places: the logits' scale bounds the difference
    assert (few - full).abs().max() <= 2.0 ** -6 * full.abs().max()
    assert (few.argmax(1) == top_ids[ids.long(), 0]).float().mean() > 0.9
    model.check()


def test_small_model_steps_are_reproducible(example):
    a, b = example.train(5), example.train(5)
    assert a[2] == b[2]
    for n in a[0].w:
        assert torch.equal(a[0].w[n], b[0].w[n]), n
