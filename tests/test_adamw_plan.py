"""An AdamW plan notices that a tensor's memory or a parameter's gradient is no longer what it was made
with, before anything is launched.  The checks run on CPU tensors here; the step that makes
them is tested on the GPU (test_gpu_adamw_plan.py)."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq


def plan(own_grads=True):
    p = [torch.nn.Parameter(torch.zeros(n)) for n in (5, 0, 300)]
    g = [torch.ones_like(t) for t in p]
    if own_grads:
        for a, b in zip(p, g):
            a.grad = b
    m, v = ([torch.zeros(t.shape) for t in p] for _ in range(2))
    return fq.AdamwPlan({"params": p, "grads": g, "m": m, "v": v}, None, 1, 0, None), p, g, m, v


def test_unchanged_tensors_pass():
    made, p, g, m, v = plan()
    made.check()
    with torch.no_grad():
        p[0].add_(1), g[2].zero_(), m[2].fill_(3)
    torch.optim.SGD(p, 0.1).zero_grad(set_to_none=False)
    made.check()


@pytest.mark.parametrize("which", range(4))
def test_other_memory(which):
    for change in (lambda t: setattr(t, "data", t.data.clone()), lambda t: t.untyped_storage().resize_(0)):
        made, *lists = plan()
        change(lists[which][2])
        with pytest.raises(ValueError, match="other memory"):
            made.check()


def test_another_gradient():
    made, p, *_ = plan()
    torch.optim.SGD(p, 0.1).zero_grad(set_to_none=True)
    with pytest.raises(ValueError, match="gradient"):
        made.check()
    (3 * p[2]).sum().backward()   # a new .grad
    with pytest.raises(ValueError, match="gradient"):
        made.check()


def test_gradients_of_their_own_do_not_follow():
    """Gradients that were nobody's .grad (buffers that the caller fills) are read whatever .grad is."""
    made, p, *_ = plan(own_grads=False)
    p[2].grad = torch.zeros(300)
    made.check()


def test_missing_lists_and_gradients():
    z = [torch.zeros(4)]
    for lists in ((None, z, z, z), (z, None, z, z), (z, z, None, z), (z, z, z, None)):
        with pytest.raises(ValueError, match="are needed"):
            fq.fp8q_adamw_plan(*lists)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        fq.fp8q_adamw_plan(z, [None], z, z)       # a parameter without a gradient
