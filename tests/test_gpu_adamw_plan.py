"""fp8q_adamw raises before it launches anything if the plan's tensors are not what they were, and runs
on where they are."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu


def made(n=1000):
    p = torch.nn.Parameter(torch.zeros(n, device="cuda"))
    p.grad = torch.ones(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    return fq.fp8q_adamw_plan([p], [p.grad], [m], [v]), p, m, v


def test_the_step_follows_gradients_filled_in_place():
    plan, p, m, v = made()
    for step in (1, 2):
        p.grad.zero_()
        (2 * p).sum().backward()      # adds into the same .grad
        fq.fp8q_adamw(plan, lr=0.5, step=step)
    torch.cuda.synchronize()
    # a gradient of 2 in both steps: m = 2 (1 - 0.81) and each step moves by lr, up to FP32's roundings
    assert bool(((m - 0.38).abs() < 1e-6).all()) and bool(((p + 1.0).abs() < 1e-5).all())


@pytest.mark.parametrize("what", ["data", "resize", "set_to_none", "new gradient"])
def test_a_stale_plan_is_refused(what):
    plan, p, m, v = made()
    old = p.data
    if what == "data":
        p.data = torch.zeros_like(p)
    elif what == "resize":
        v.untyped_storage().resize_(0)
    else:
        p.grad = None
        if what == "new gradient":
            p.sum().backward()
    with pytest.raises(ValueError, match="make a new plan"):
        fq.fp8q_adamw(plan, lr=0.5)
    torch.cuda.synchronize()
    assert not bool(old.any()) and not bool(m.any())
    if what in ("data", "new gradient"):
        fq.fp8q_adamw(fq.fp8q_adamw_plan([p], [p.grad], [m], [v]), lr=0.5)
        assert bool(p.any())
