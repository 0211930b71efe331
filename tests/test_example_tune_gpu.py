"""Tuning in the example: the KL term's reference is the model that tuning began with, on every batch."""
import importlib.util
import os

import pytest
import torch

from lm_testlib import setup

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    setup()
    spec = importlib.util.spec_from_file_location("distill_student", os.path.join(ROOT, "examples", "distill_student.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("mix", [False, True])
def test_the_reference_stays(example, mix, capsys):
    T, V = 128, 200
    starts = torch.arange(0, T + 1, 32, dtype=torch.int32, device="cuda") if mix else None
    student = example.Student(T, V, 128, 512, layers=2, k=8, mix=mix, starts=starts)
    weight = torch.full((T,), 1.0 / T, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    began, calls = {n: p.clone() for n, p in student.p.items()}, []
    step = student.policy_and_gradients

    def recorded(tokens, sampled, old, ref, *rest):
        calls.append((tokens, sampled, old.clone(), ref.clone()))
        return step(tokens, sampled, old, ref, *rest)

    student.policy_and_gradients = recorded
    example.tune(student, 5, weight, g)
    assert len(calls) == 5
    assert torch.equal(calls[0][2], calls[0][3])     # nothing has moved yet
    for tokens, sampled, old, ref in calls[2:]:
        assert not torch.equal(old, ref)
        assert torch.equal(ref, student.log_probabilities(tokens, sampled, weight, began))
