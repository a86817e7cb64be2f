"""The operators together, as the example trains with them (-m gpu)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_loss(model, flat, ids, targets):
    """The example's model in elementary fp32 operations on the same bf16 parameters."""
    w = model.views(flat)
    norm = lambda v, s: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-5) * s  # noqa: E731
    r = w["embed"][ids] * model.dim ** 0.5
    z = norm(r, w["pre0"])
    for l in range(model.layers):
        gu = z @ w["up%d" % l].t()
        g, u = gu[:, :model.hidden], gu[:, model.hidden:]
        y = (g * torch.sigmoid(g) * u) @ w["down%d" % l].t()
        r = r + w["gate%d" % l] * norm(y, w["post%d" % l])
        z = norm(r, w["pre%d" % (l + 1)])
    return torch.nn.functional.cross_entropy(z @ w["embed"].t(), targets)


@pytest.mark.parametrize("vocab,dim,hidden,layers,tokens", [(300, 64, 176, 2, 512), (101, 40, 72, 1, 77)])
def test_gradients_of_a_model(dev, vocab, dim, hidden, layers, tokens):
    """Every parameter's gradient within 3 percent (in norm) of automatic differentiation in fp32.  What is between them: bf16
    activations and gradients (2^-9 each, through 10 or so stages) and 8-bit checkpoints, whose values are off by up to half a
    step in 64 (root mean square about 0.5 percent of a value)."""
    import gated_mlp_lm as ex
    model = ex.Model(vocab, dim, hidden, layers, tokens)
    flat = model.init(5).bfloat16()
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids, targets = ex.batch(vocab, tokens, gen)
    grads = torch.zeros(model.psi, dtype=torch.bfloat16, device="cuda")
    loss = model.forward_backward(flat, grads, ids, targets, 64.0)
    ref = flat.float().requires_grad_()
    want_loss = plain_loss(model, ref, ids, targets)
    want, = torch.autograd.grad(want_loss, ref)
    assert abs(float(loss) - float(want_loss)) < 0.02 * float(want_loss)
    got, want = model.views(grads.float() / 64.0), model.views(want)
    for k in want:
        off = float((got[k] - want[k]).norm() / want[k].norm())
        assert off < 0.03, (k, off)


def test_training_learns_the_rule(dev):
    import gated_mlp_lm as ex
    losses, (skipped, error) = ex.train(steps=40, layers=2, dim=128, hidden=352, vocab=200, tokens=1024)
    assert not skipped and not error
    assert losses[0] > 4.5 and losses[-1] < 0.5 * losses[0], losses


def test_overflow_skips_the_step(dev):
    """A weight that overflows the activations: the checkpoints carry that on as NaNs, and the step is skipped."""
    import gated_mlp_lm as ex
    import zero_gradient_sync_gb300 as dp
    from zero_gradient_sync_gb300.buffers import StepBuffers
    model = ex.Model(50, 64, 96, 1, 128)
    bufs = StepBuffers(dp.Layout.even(model.psi, 1, stage=1), 1)
    start = model.init()
    model.views(start)["up0"][3, 5] = 3e38
    bufs.master[0].copy_(start)
    bufs.replicas[0].copy_(start)
    bufs.grads[0].zero_()
    gen = torch.Generator(device="cuda").manual_seed(1)
    model.forward_backward(bufs.replicas[0], bufs.grad(0, 0), *ex.batch(50, 128, gen), 1.0)
    assert not torch.isfinite(bufs.grads[0].float()).all()
    bufs.step(dp.adam(), 1.0)
    assert bufs.status() == (1, 0)
    assert torch.equal(bufs.master[0], start)
