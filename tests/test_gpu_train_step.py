"""The operators together, in examples/train_step.py: one training step's loss
and gradients against the same model differentiated in 64 bits (with the
routing the GPU chose), the clipping, single-token scoring, and a falling loss.

Tolerance: every activation and gradient between two operators is rounded to
bf16 (RMS relative error 2^-9.2 each); a gradient has some twenty such
roundings behind it, of random signs, and sums that may cancel to a third of
their terms: 20^(1/2) 2^-9.2 3 = 2.3e-2, held to 5e-2.  The loss is a mean
over the tokens of logits with half as many."""
import importlib.util
import os

import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    _build.build()
    moe.load()
    spec = importlib.util.spec_from_file_location(
        "train_step_example", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(model, ids, labels):
    """Mean loss and the gradients of every parameter, in 64 bits."""
    p = {k: v.double().cpu().requires_grad_() for k, v in model.params.items()}
    ids, labels = ids.cpu().long(), labels.cpu().long()

    def norm(x, w):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    r = p["embed"][ids.clamp(min=0)] * (ids >= 0).double()[:, None]
    n = norm(r, p["pre0"])
    for i in range(model.L):
        logits = n @ p[f"router{i}"].t()
        top = model.topk[i].cpu().long()
        w = torch.softmax(logits.gather(1, top), 1)
        y = torch.zeros_like(n)
        for e in range(model.E):
            h = n @ p[f"w1_{i}"][e].t()
            h = torch.nn.functional.silu(h[:, :model.F]) * h[:, model.F:]
            y = y + (w * (top == e)).sum(1, keepdim=True) * (h @ p[f"w2_{i}"][e].t())
        r = r + p[f"gate{i}"] * norm(y, p[f"post{i}"])
        n = norm(r, p[f"pre{i + 1}"])
    z = n @ p["head"].t()
    valid = labels >= 0
    loss = (torch.logsumexp(z, 1) - z.gather(1, labels.clamp(min=0)[:, None])[:, 0])[valid].sum() \
        / valid.sum()
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("T", [96, 300])
def test_step_against_64_bits(example, T):
    model = example.MoELM(vocab=333, layers=2)
    ids, labels = example.batch(T, model.V, torch.Generator().manual_seed(T))
    ids[5], labels[3], labels[T - 1] = -1, -1, -100  # a padded token, masked labels
    valid = (labels >= 0).sum().float()
    loss = float(model.forward(ids, labels).sum() / valid)
    model.backward(ids, labels, (1 / valid).expand(T).contiguous(), max_norm=float("inf"))
    assert model.status() == moe.MOE_OK
    want, grads = reference(model, ids, labels)
    assert abs(loss - want) <= 1e-2 * abs(want)
    total = 0.0
    for k, g in grads.items():
        d = model.grads[k].double().cpu() - g
        assert float(d.norm()) <= 5e-2 * float(g.norm()), (k, float(d.norm() / g.norm()))
        total += float((model.grads[k].double() ** 2).sum())
    assert abs(float(model.norm[0]) - total ** 0.5) <= 1e-4 * total ** 0.5
    # the same step clipped: the gradients scaled, to a norm of a tenth
    free = {k: v.clone() for k, v in model.grads.items()}
    limit = 0.1 * total ** 0.5
    model.backward(ids, labels, (1 / valid).expand(T).contiguous(), max_norm=limit)
    for k, v in model.grads.items():
        assert (v.double() - 0.1 * free[k].double()).norm() <= 5e-3 * (0.1 * free[k].double()).norm()


def test_single_tokens_score_as_in_the_batch(example):
    """The model has no attention, so a token's loss does not depend on its neighbours."""
    model = example.MoELM(vocab=500, layers=1)
    ids, labels = example.batch(40, model.V, torch.Generator().manual_seed(3))
    whole = model.forward(ids, labels).clone()
    one = torch.stack([model.forward(ids[t:t + 1], labels[t:t + 1])[0].clone() for t in range(40)])
    assert (one - whole).abs().max() <= 2e-2 * whole.abs().max()


def test_loss_falls(example):
    model = example.MoELM(vocab=100, layers=1)
    g = torch.Generator().manual_seed(7)
    first = last = None
    for i in range(60):
        loss = float(model.step(*example.batch(512, model.V, g), lr=1.0))
        first, last = (loss if i == 0 else first), loss
    assert model.status() == moe.MOE_OK
    assert last < 0.75 * first, (first, last)
