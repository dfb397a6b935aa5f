"""Argument checks of the MoE training-step entry points and of AdamW, without a GPU: the C
entry points reject bad arguments before any HIP call, and the binding refuses CPU tensors,
wrong shapes and shared memory."""
import ctypes
import math
import os
import re

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a fake, 16-byte aligned device address (never dereferenced)
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return fq.load_library()


@pytest.fixture(scope="module")
def E():
    text = open(os.path.join(ROOT, "include", "fp8q.h")).read()
    return {k: int(v) for k, v in re.findall(r"\b(FP8Q_[A-Z0-9_]+)\s*=\s*(-?\d+)", text)}


def check(f, base, E, cases):
    """`base`: arguments of a valid call by name, in order; cases: (changes, status)."""
    for change, status in cases:
        args = {**base, **change}
        assert f(*args.values()) == E[status], (change, status)


def test_sort(lib, E):
    base = dict(ids=A, T=4, k=8, e0=0, E=32, x=A, dt=0, H=64, cap=32, xs=A, off=A, tr=A, rt=A, stream=None)
    check(lib.fp8q_moe_sort, base, E, [
        (dict(dt=2), "FP8Q_ERR_DTYPE"), (dict(H=60), "FP8Q_ERR_SHAPE"), (dict(H=-8), "FP8Q_ERR_SHAPE"),
        (dict(k=0), "FP8Q_ERR_SHAPE"), (dict(k=65), "FP8Q_ERR_SHAPE"), (dict(E=0), "FP8Q_ERR_SHAPE"),
        (dict(E=1025), "FP8Q_ERR_SHAPE"), (dict(e0=-1), "FP8Q_ERR_SHAPE"), (dict(cap=-1), "FP8Q_ERR_SHAPE"),
        (dict(T=-1), "FP8Q_ERR_SHAPE"), (dict(T=BIG), "FP8Q_ERR_SHAPE"), (dict(T=1 << 28, k=8), "FP8Q_ERR_SHAPE"),
        (dict(T=1 << 27, k=1, H=1 << 17), "FP8Q_ERR_SHAPE"),      # more workgroups than a grid holds
        (dict(ids=0), "FP8Q_ERR_NULL"), (dict(x=0), "FP8Q_ERR_NULL"), (dict(xs=0), "FP8Q_ERR_NULL"),
        (dict(off=0), "FP8Q_ERR_NULL"), (dict(tr=0), "FP8Q_ERR_NULL"), (dict(rt=0), "FP8Q_ERR_NULL"),
        (dict(x=A + 8), "FP8Q_ERR_ALIGN"), (dict(xs=A + 4), "FP8Q_ERR_ALIGN"), (dict(ids=A + 2), "FP8Q_ERR_ALIGN"),
        (dict(off=A + 1), "FP8Q_ERR_ALIGN"), (dict(rt=A + 3), "FP8Q_ERR_ALIGN")])


def test_sort_backward(lib, E):
    base = dict(dxs=A, dt=0, cap=32, H=64, tr=A, T=4, k=8, dx=A, out=1, stream=None)
    check(lib.fp8q_moe_sort_backward, base, E, [
        (dict(dt=3), "FP8Q_ERR_DTYPE"), (dict(out=-1), "FP8Q_ERR_DTYPE"), (dict(H=12), "FP8Q_ERR_SHAPE"),
        (dict(k=65), "FP8Q_ERR_SHAPE"), (dict(cap=BIG), "FP8Q_ERR_SHAPE"), (dict(T=0, tr=0, dx=0, dxs=0), "FP8Q_OK"),
        (dict(H=0, dx=0), "FP8Q_OK"), (dict(tr=0), "FP8Q_ERR_NULL"), (dict(dx=0), "FP8Q_ERR_NULL"),
        (dict(dxs=0), "FP8Q_ERR_NULL"), (dict(dxs=A + 8), "FP8Q_ERR_ALIGN"), (dict(dx=A + 2), "FP8Q_ERR_ALIGN")])


def test_combine_backward(lib, E):
    base = dict(dy=A, dydt=0, out=A, dt=0, cap=32, N=64, tr=A, w=A, T=4, k=8, dout=A, dw=A, stream=None)
    check(lib.fp8q_moe_combine_backward, base, E, [
        (dict(dydt=2), "FP8Q_ERR_DTYPE"), (dict(dt=2), "FP8Q_ERR_DTYPE"), (dict(N=4), "FP8Q_ERR_SHAPE"),
        (dict(k=0), "FP8Q_ERR_SHAPE"), (dict(T=-4), "FP8Q_ERR_SHAPE"), (dict(T=0, dy=0, tr=0, w=0, dw=0), "FP8Q_OK"),
        (dict(dy=0), "FP8Q_ERR_NULL"), (dict(out=0), "FP8Q_ERR_NULL"), (dict(tr=0), "FP8Q_ERR_NULL"),
        (dict(w=0), "FP8Q_ERR_NULL"), (dict(dout=0), "FP8Q_ERR_NULL"), (dict(dw=0), "FP8Q_ERR_NULL"),
        (dict(dy=A + 4), "FP8Q_ERR_ALIGN"), (dict(dout=A + 8), "FP8Q_ERR_ALIGN"), (dict(dw=A + 2), "FP8Q_ERR_ALIGN")])


def test_swiglu_backward(lib, E):
    base = dict(gu=A, dh=A, dt=0, M=4, I=64, dgu=A, h=0, stream=None)
    check(lib.fp8q_swiglu_backward, base, E, [
        (dict(dt=7), "FP8Q_ERR_DTYPE"), (dict(I=12), "FP8Q_ERR_SHAPE"), (dict(M=-1), "FP8Q_ERR_SHAPE"),
        (dict(M=(1 << 31) - 1, I=(1 << 31) - 8), "FP8Q_ERR_SHAPE"), (dict(M=0, gu=0), "FP8Q_OK"),
        (dict(I=0, dgu=0), "FP8Q_OK"), (dict(gu=0), "FP8Q_ERR_NULL"), (dict(dh=0), "FP8Q_ERR_NULL"),
        (dict(dgu=0), "FP8Q_ERR_NULL"), (dict(h=A + 2), "FP8Q_ERR_ALIGN"), (dict(dh=A + 8), "FP8Q_ERR_ALIGN")])


def test_quantize_act_grouped(lib, E):
    base = dict(x=A, off=A, G=4, M=100, K=256, xq=A, sa=A, xqt=A, sat=A, stream=None)
    check(lib.fp8q_quantize_act_grouped, base, E, [
        (dict(G=0), "FP8Q_ERR_SHAPE"), (dict(K=200), "FP8Q_ERR_SHAPE"), (dict(M=-1), "FP8Q_ERR_SHAPE"),
        (dict(M=(1 << 31) - 1, K=1 << 20), "FP8Q_ERR_SHAPE"), (dict(G=BIG - 1, K=1 << 20), "FP8Q_ERR_SHAPE"),
        (dict(M=0, x=0, off=0, xq=0, sa=0, xqt=0, sat=0), "FP8Q_OK"), (dict(K=0, x=0), "FP8Q_OK"),
        (dict(x=0), "FP8Q_ERR_NULL"), (dict(off=0), "FP8Q_ERR_NULL"), (dict(xqt=0), "FP8Q_ERR_NULL"),
        (dict(sat=0), "FP8Q_ERR_NULL"), (dict(xq=0), "FP8Q_ERR_NULL"), (dict(sa=0), "FP8Q_ERR_NULL"),
        (dict(x=A + 2), "FP8Q_ERR_ALIGN"), (dict(off=A + 2), "FP8Q_ERR_ALIGN"), (dict(xqt=A + 8), "FP8Q_ERR_ALIGN")])


def test_grouped_gemm_rowscaled(lib, E):
    base = dict(a=A, sa=A, b=A, sb=A, off=A, G=4, M=100, P=128, Q=256, c=A, dt=1, stream=None)
    check(lib.fp8q_grouped_gemm_rowscaled, base, E, [
        (dict(dt=4), "FP8Q_ERR_DTYPE"), (dict(G=0), "FP8Q_ERR_SHAPE"), (dict(P=100), "FP8Q_ERR_SHAPE"),
        (dict(Q=-128), "FP8Q_ERR_SHAPE"), (dict(M=BIG), "FP8Q_ERR_SHAPE"), (dict(P=(1 << 22) + 128), "FP8Q_ERR_SHAPE"),
        (dict(G=1 << 20, P=1 << 20, Q=1 << 20), "FP8Q_ERR_SHAPE"), (dict(P=0, c=0), "FP8Q_OK"),
        (dict(Q=0, a=0), "FP8Q_OK"), (dict(a=0), "FP8Q_ERR_NULL"), (dict(sb=0), "FP8Q_ERR_NULL"),
        (dict(off=0), "FP8Q_ERR_NULL"), (dict(c=0), "FP8Q_ERR_NULL"), (dict(M=0, a=0, c=0), "FP8Q_ERR_NULL"),
        (dict(b=A + 8), "FP8Q_ERR_ALIGN"), (dict(off=A + 2), "FP8Q_ERR_ALIGN"), (dict(c=A + 4), "FP8Q_ERR_ALIGN")])


def test_adamw(lib, E):
    def call(count=1, grad=1, state=0, tensors=True, hyper=True, tensor=(), **change):
        t = (fq._AdamwTensor * 1)(fq._AdamwTensor(A, A, A, A, A, A, 0, 100))
        for name, value in dict(tensor).items():
            setattr(t[0], name, value)
        h = fq._AdamwHyper(1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 1, None)
        for name, value in change.items():
            setattr(h, name, value)
        return lib.fp8q_adamw(t if tensors else None, count, grad, state, ctypes.byref(h) if hyper else None, None)

    for bad in (dict(grad=2), dict(state=2), dict(state=-1)):
        assert call(**bad) == E["FP8Q_ERR_DTYPE"]
    for bad in (dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5), dict(eps=-1e-8),
                dict(eps=math.nan), dict(step=0), dict(step=-3), dict(weight_decay=math.inf), dict(grad_scale=math.nan)):
        assert call(**bad) == E["FP8Q_ERR_VALUE"], bad
    assert "hyperparameter" in fq.status_string(E["FP8Q_ERR_VALUE"])
    assert call(count=-1) == E["FP8Q_ERR_SHAPE"]
    assert call(tensor=dict(n=-1)) == E["FP8Q_ERR_SHAPE"] == call(tensor=dict(n=1 << 40))
    assert call(tensors=False) == E["FP8Q_ERR_NULL"] == call(hyper=False)
    for name in ("p", "grad", "m", "v"):
        assert call(tensor={name: None}) == E["FP8Q_ERR_NULL"]
        assert call(tensor={name: A + 8}) == E["FP8Q_ERR_ALIGN"]
    for name in ("m_scale", "v_scale"):
        assert call(state=1, tensor={name: None}) == E["FP8Q_ERR_NULL"]
        assert call(state=1, tensor={name: A + 2}) == E["FP8Q_ERR_ALIGN"]
    assert call(tensor=dict(p_bf16=A + 2)) == E["FP8Q_ERR_ALIGN"] == call(scalars=A + 2)
    assert call(count=0, tensors=False) == E["FP8Q_OK"] == call(tensor=dict(n=0, p=None))


def test_binding_refuses_cpu_tensors_and_other_types():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_moe_sort(z((4, 2), dtype=torch.int32), z(4, 8), 0, 4)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        fq.fp8q_moe_sort_backward(z((4, 8), dtype=torch.float16), z((4, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_moe_combine_backward(z(4, 8), z(4, 8), z((4, 1), dtype=torch.int32), z(4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_swiglu_backward(z((4, 16), dtype=torch.bfloat16), z(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_quantize_act_grouped(z((4, 128), dtype=torch.bfloat16), z(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_grouped_gemm_rowscaled(*[z((1, 128, 128), dtype=torch.uint8)] * 4, z(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_adamw_plan([z(4)], [z(4)], [z(4)], [z(4)])
    with pytest.raises(ValueError, match="1 tensors each"):
        fq.fp8q_adamw_plan([z(4)], [], [z(4)], [z(4)])
    with pytest.raises(ValueError, match="go together"):
        fq.fp8q_adamw_plan([z(4)], [z(4)], [z(4)], [z(4)], m_scales=[z(1)])
    with pytest.raises(ValueError, match="plan"):
        fq.fp8q_adamw([z(4)], lr=1e-3)
