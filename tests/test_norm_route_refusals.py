"""Argument checks of the norm and of the router, without a GPU: the C entry points reject bad arguments
before any HIP call, and the binding refuses CPU tensors, wrong shapes and wrong types."""
import math
import os
import re

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a fake, 16-byte aligned device address (never dereferenced)
BIG = 1 << 31
E = {k: int(v) for k, v in re.findall(r"\b(FP8Q_[A-Z0-9_]+)\s*=\s*(-?\d+)", open(os.path.join(ROOT, "include", "fp8q.h")).read())}


@pytest.fixture(scope="module")
def lib():
    return fq.load_library()


def check(f, base, cases):
    """`base`: arguments of a valid call by name, in order; cases: (changes, status)."""
    for change, status in cases:
        assert set(change) <= set(base)
        assert f(*{**base, **change}.values()) == E[status], (change, status)


SHAPES = [dict(H=12), dict(H=0), dict(H=-8), dict(H=16392), dict(T=-1), dict(T=BIG)]


def test_layer_norm(lib):
    base = dict(x=A, xdt=0, w=A, b=A, T=4, H=64, eps=1e-5, center=1, y=A, ydt=1, mean=A, rstd=A, stream=None)
    check(lib.fp8q_layer_norm, base, [(s, "FP8Q_ERR_SHAPE") for s in SHAPES] + [
        (dict(xdt=2), "FP8Q_ERR_DTYPE"), (dict(ydt=-1), "FP8Q_ERR_DTYPE"), (dict(eps=-1e-9), "FP8Q_ERR_VALUE"),
        (dict(eps=math.nan), "FP8Q_ERR_VALUE"), (dict(eps=1e39), "FP8Q_ERR_VALUE"),
        (dict(T=0, x=0, w=0, b=0, y=0, mean=0, rstd=0), "FP8Q_OK"), (dict(x=0), "FP8Q_ERR_NULL"),
        (dict(w=0), "FP8Q_ERR_NULL"), (dict(y=0), "FP8Q_ERR_NULL"), (dict(mean=0), "FP8Q_ERR_NULL"),
        (dict(rstd=0), "FP8Q_ERR_NULL"), (dict(x=A + 8), "FP8Q_ERR_ALIGN"), (dict(w=A + 4), "FP8Q_ERR_ALIGN"),
        (dict(b=A + 4), "FP8Q_ERR_ALIGN"), (dict(y=A + 8), "FP8Q_ERR_ALIGN"), (dict(mean=A + 2), "FP8Q_ERR_ALIGN"),
        (dict(rstd=A + 1), "FP8Q_ERR_ALIGN")])


def test_layer_norm_backward(lib):
    base = dict(dy=A, dydt=0, x=A, xdt=1, w=A, mean=A, rstd=A, T=4, H=64, dx=A, dxdt=0, dw=A, db=A, ws=A, stream=None)
    check(lib.fp8q_layer_norm_backward, base, [(s, "FP8Q_ERR_SHAPE") for s in SHAPES] + [
        (dict(dydt=2), "FP8Q_ERR_DTYPE"), (dict(xdt=2), "FP8Q_ERR_DTYPE"), (dict(dxdt=2), "FP8Q_ERR_DTYPE"),
        *[({name: 0}, "FP8Q_ERR_NULL") for name in ("dy", "x", "w", "rstd", "dx", "dw", "ws")],
        *[({name: A + 8}, "FP8Q_ERR_ALIGN") for name in ("dy", "x", "w", "dx", "ws")],
        *[({name: A + 2}, "FP8Q_ERR_ALIGN") for name in ("mean", "rstd", "dw", "db")]])
    assert lib.fp8q_layer_norm_backward_workspace(4, 12) == E["FP8Q_ERR_SHAPE"]
    assert lib.fp8q_layer_norm_backward_workspace(0, 64) == 0
    assert lib.fp8q_layer_norm_backward_workspace(5, 64) == 2 * 8 * 64
    assert lib.fp8q_layer_norm_backward_workspace(BIG - 1, 16384) == 2048 * 16384


BAD_ROUTES = [dict(B=0), dict(B=65536), dict(S=-1), dict(S=BIG), dict(E=0), dict(E=1025), dict(k=0), dict(k=65, E=256),
              dict(k=9, E=8), dict(B=8, S=1 << 26, k=4)]


def test_moe_route(lib):
    base = dict(z=A, dt=1, B=2, S=5, E=16, k=4, bias=A, valid=A, score=0, norm=1, scale=1.0, balance=1e-3, ids=A, w=A, counts=A,
                loss=A, slope=A, ws=A, stream=None)
    check(lib.fp8q_moe_route, base, [(s, "FP8Q_ERR_SHAPE") for s in BAD_ROUTES] + [
        (dict(dt=2), "FP8Q_ERR_DTYPE"), (dict(score=2), "FP8Q_ERR_DTYPE"),
        *[(dict(scale=v), "FP8Q_ERR_VALUE") for v in (0.0, -1.0, math.nan, math.inf, 1e39, 1e-39, 1e-60)],
        (dict(balance=math.nan), "FP8Q_ERR_VALUE"), (dict(balance=math.inf), "FP8Q_ERR_VALUE"),
        *[({name: 0}, "FP8Q_ERR_NULL") for name in ("z", "ids", "w", "counts", "loss", "slope", "ws")],
        (dict(z=A + 8), "FP8Q_ERR_ALIGN"), (dict(ws=A + 8), "FP8Q_ERR_ALIGN"),
        *[({name: A + 2}, "FP8Q_ERR_ALIGN") for name in ("bias", "ids", "w", "counts", "loss", "slope")]])
    assert lib.fp8q_moe_route_workspace(0, 5, 16) == E["FP8Q_ERR_SHAPE"] == lib.fp8q_moe_route_workspace(1, 5, 1025)
    assert lib.fp8q_moe_route_workspace(3, 0, 16) > 0


def test_moe_route_backward(lib):
    base = dict(z=A, dt=0, B=2, S=5, E=16, k=4, ids=A, w=A, dw=A, slope=A, dloss=A, score=1, norm=0, scale=2.5, dz=A, dzdt=1,
                stream=None)
    check(lib.fp8q_moe_route_backward, base, [(s, "FP8Q_ERR_SHAPE") for s in BAD_ROUTES] + [
        (dict(dt=2), "FP8Q_ERR_DTYPE"), (dict(dzdt=2), "FP8Q_ERR_DTYPE"), (dict(score=-1), "FP8Q_ERR_DTYPE"),
        *[(dict(scale=v), "FP8Q_ERR_VALUE") for v in (0.0, -1.0, math.nan, 1e-39)],
        (dict(S=0, z=0, ids=0, w=0, dw=0, slope=0, dz=0), "FP8Q_OK"),
        *[({name: 0}, "FP8Q_ERR_NULL") for name in ("z", "ids", "w", "dw", "slope", "dz")],
        (dict(z=A + 8), "FP8Q_ERR_ALIGN"), (dict(dz=A + 4), "FP8Q_ERR_ALIGN"),
        *[({name: A + 2}, "FP8Q_ERR_ALIGN") for name in ("ids", "w", "dw", "slope", "dloss")]])


def test_binding_refuses_cpu_tensors_and_other_types():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_layer_norm(z(4, 8), z(8))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        fq.fp8q_layer_norm(z((4, 8), dtype=torch.float16), z(8))
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_layer_norm_backward(z(4, 8), z(4, 8), z(8), z(4), z(4))
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_moe_route(z(4, 8), 2)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        fq.fp8q_moe_route(z((4, 8), dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_moe_route_backward(z(4, 8), z((4, 2), dtype=torch.int32), z(4, 2), z(4, 2), z(8))
