"""The model operators together: examples/distill_student.py trains, and the
gradients that its first pass writes to a rank's flat buffer agree with those of
the same model in fp32 (torch autograd).  Activations and gradients of the
example are bf16 (half an ulp is 2^-9 to 2^-8 of a value) and
pass about ten roundings one after the other, which add as random errors do:
2^-8 * sqrt(10) = 0.012 of a tensor's norm, times 3 for the chains' differing
lengths."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import distill_student
    return distill_student


def test_student_learns(example):
    loss = example.run(30)
    assert all(x == x for x in loss)
    assert loss[-1] < 0.8 * loss[0]


def test_gradients_agree_with_autograd(example):
    E = example
    student, (ids, (tl, ti), labels) = E.Student(), E.Teacher().batch()
    logits, kept = student.forward(ids)
    student.backward(ids, logits, kept, (tl, ti), labels, student.grads[0])
    got = E.views(student.grads[0])

    w = {k: v.float().clone().requires_grad_() for k, v in student.w.items()}

    def norm(x, weight):
        return x * torch.rsqrt((x * x).mean(1, keepdim=True) + E.NORM["eps"]) * weight

    x = w["table"][ids] * student.scale
    u = norm(x, w["first_norm"])
    for b in range(E.BLOCKS):
        h = torch.relu(u @ w["up%d" % b].t()) @ w["down%d" % b].t()
        x = x + E.NORM["branch_scale"] * w["gate%d" % b] * norm(h, w["post%d" % b])
        u = norm(x, w["pre%d" % b])
    out = u @ w["table"].t()
    p = torch.softmax(tl / E.TEMPERATURE, 1)
    q = torch.log_softmax(out / E.TEMPERATURE, 1)
    kl = (p * (torch.log(p) - torch.gather(q, 1, ti.long()))).sum(1) * E.TEMPERATURE ** 2
    ce = torch.nn.functional.cross_entropy(out, labels, ignore_index=-100, reduction="sum")
    ((E.CE_WEIGHT * ce + E.KL_WEIGHT * kl.sum()) / E.TOKENS).backward()
    for name, g in got.items():
        want = w[name].grad
        error = float((g.float() - want).norm() / want.norm())
        assert error <= 3 * 2.0 ** -8 * 10 ** 0.5, (name, error)
