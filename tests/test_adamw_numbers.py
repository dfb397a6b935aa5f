"""fp8q_adamw takes its numbers as doubles and computes in FP32: what FP32 cannot hold is refused, on
the host, before any launch.  No GPU: the pointers are fake, and a call that passes its checks ends
at the missing device."""
import ctypes
import os
import re

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

A = 1 << 20  # a fake, 16-byte aligned device address (never dereferenced)
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8q.h")
E = {k: int(v) for k, v in re.findall(r"\b(FP8Q_[A-Z0-9_]+)\s*=\s*(-?\d+)", open(HEADER).read())}


def step(state=0, **change):
    t = (fq._AdamwTensor * 1)(fq._AdamwTensor(A, A, A, A, A, A, 0, 100))
    h = fq._AdamwHyper(1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 1, None)
    for name, value in change.items():
        setattr(h, name, value)
    return fq.load_library().fp8q_adamw(t, 1, 1, state, ctypes.byref(h), None)


@pytest.mark.parametrize("state", [0, 1])
@pytest.mark.parametrize("change", [
    dict(lr=1e300), dict(lr=-1e39), dict(weight_decay=1e60), dict(grad_scale=3.5e38),      # inf in FP32
    dict(eps=1e-50), dict(grad_scale=1e-46), dict(lr=1e-60), dict(beta1=1e-300),           # 0 in FP32
    dict(beta1=1 - 1e-12), dict(beta2=1 - 1e-9),                                           # 1 in FP32
    dict(lr=1e38, beta1=0.999), dict(lr=1e30, weight_decay=1e10)])                         # inf on the way
def test_numbers_that_fp32_does_not_hold(change, state):
    assert step(state, **change) == E["FP8Q_ERR_VALUE"]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would run on fake addresses")
@pytest.mark.parametrize("change", [
    dict(lr=0.0), dict(lr=-1e-3), dict(eps=0.0), dict(eps=1e-45), dict(weight_decay=0.0), dict(grad_scale=0.0), dict(grad_scale=-1.0),
    dict(beta1=0.0, beta2=0.0), dict(beta1=1 - 2.0 ** -24, beta2=1 - 2.0 ** -24), dict(lr=3.4e38, beta1=0.0),
    dict(step=2 ** 62), dict(lr=1e38, beta1=0.999, scalars=A)])
def test_numbers_that_it_holds(change):
    assert step(**change) == E["FP8Q_ERR_DEVICE"]
