"""Argument checks of the orthogonalized matrices and of Muon, without a GPU."""
import ctypes
import math
import os
import re

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a fake, 16-byte aligned device address (never dereferenced)
E = {k: int(v) for k, v in re.findall(r"\b(FP8Q_[A-Z0-9_]+)\s*=\s*(-?\d+)", open(os.path.join(ROOT, "include", "fp8q.h")).read())}


def ns(**change):
    values = {"a": 3.4, "b": -4.7, "c": 2.0, "steps": 5, **change}
    return fq._NewtonSchulz(*values.values())


def orthogonalize(x=A, dt=0, G=2, P=8, Q=16, out=A, ws=A, hyper=True, **change):
    n = ns(**change)
    return fq.load_library().fp8q_orthogonalize(x, dt, G, P, Q, ctypes.byref(n) if hyper else None, out, ws, None)


def muon(p=A, g=A, dt=1, m=A, G=2, P=8, Q=16, copy=0, ws=A, given=True, device_lr=None, numbers=None, **change):
    values = {"lr": 1e-3, "beta": 0.95, "weight_decay": 0.1, "scale": 1.0, "grad_scale": 1.0, **(numbers or {})}
    h = fq._MuonHyper(*values.values(), ns(**change), 1, device_lr)
    return fq.load_library().fp8q_muon(p, g, dt, m, G, P, Q, ctypes.byref(h) if given else None, copy, ws, None)


BOTH = pytest.mark.parametrize("call", [orthogonalize, muon])


@BOTH
def test_shapes_types_and_steps(call):
    for bad in (dict(G=0), dict(G=-1), dict(P=-1), dict(Q=-8), dict(P=(1 << 20) + 1), dict(Q=1 << 21), dict(G=65536),
                dict(G=60000, P=1 << 16, Q=1 << 16), dict(P=1 << 20, Q=1 << 20)):
        assert call(**bad) == E["FP8Q_ERR_SHAPE"], bad
        shape = {"G": 2, "P": 8, "Q": 16, **bad}
        assert fq.load_library().fp8q_muon_workspace(*shape.values()) == E["FP8Q_ERR_SHAPE"]
    assert call(dt=2) == E["FP8Q_ERR_DTYPE"]
    for bad in (dict(steps=0), dict(steps=-1), dict(steps=101), dict(a=math.nan), dict(b=math.inf), dict(c=1e39)):
        assert call(**bad) == E["FP8Q_ERR_VALUE"], bad
    assert call(ws=0) == E["FP8Q_ERR_NULL"]
    assert call(ws=A + 8) == E["FP8Q_ERR_ALIGN"]
    assert call(P=0, ws=0) == E["FP8Q_OK"] == call(Q=0, ws=0)


def test_orthogonalize():
    assert orthogonalize(x=0) == orthogonalize(out=0) == orthogonalize(hyper=False) == E["FP8Q_ERR_NULL"]
    assert orthogonalize(x=A + 8) == orthogonalize(out=A + 2) == E["FP8Q_ERR_ALIGN"]


def test_muon():
    assert muon(p=0) == muon(g=0) == muon(m=0) == muon(given=False) == E["FP8Q_ERR_NULL"]
    assert muon(p=A + 8) == muon(g=A + 2) == muon(m=A + 4) == muon(copy=A + 2) == muon(device_lr=A + 2) == E["FP8Q_ERR_ALIGN"]
    for bad in (dict(lr=math.nan), dict(lr=1e39), dict(beta=1.0), dict(beta=-0.1), dict(beta=1 - 1e-12), dict(scale=math.inf),
                dict(weight_decay=math.nan), dict(grad_scale=math.inf), dict(lr=1e30, scale=1e30), dict(lr=-1e30, weight_decay=1e30)):
        assert muon(numbers=bad) == E["FP8Q_ERR_VALUE"], bad


def test_workspace():
    size = fq.load_library().fp8q_muon_workspace
    assert size(1, 0, 5) == 0
    assert size(1, 300, 1000) == size(1, 1000, 300)
    # X in FP16 twice and its E4M3 rests, two square matrices, a diagonal, pairs and the sums, each rounded up to 256 bytes
    assert size(3, 128, 256) == 3 * (5 * 128 * 256 + 4 * 128 * 128) + 3 * 12 * 128 + 256


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_orthogonalize(z)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_muon(z, z, z, lr=0.1)
