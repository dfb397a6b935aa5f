"""A grid of HIP has fewer than 2^32 threads (workgroups times threads of a workgroup).  The
calls of the MoE training step and AdamW refuse what would need more, before their first launch;
the largest sizes below the bound pass the check.  No GPU: the pointers are fake, and a call that
passes its checks ends at the missing device."""
import ctypes
import os
import re

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

A = 1 << 20  # a fake, 16-byte aligned device address (never dereferenced)
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8q.h")
E = {k: int(v) for k, v in re.findall(r"\b(FP8Q_[A-Z0-9_]+)\s*=\s*(-?\d+)", open(HEADER).read())}

BOUND = 1 << 24  # workgroups of 256 threads


def sort(T, k=1, H=8, dt=0):
    return fq.load_library().fp8q_moe_sort(A, T, k, 0, 32, A, dt, H, 64, A, A, A, A, None)


def sort_backward(T, H=8):
    return fq.load_library().fp8q_moe_sort_backward(A, 0, 64, H, A, T, 1, A, 1, None)


def combine_backward(T, k):
    return fq.load_library().fp8q_moe_combine_backward(A, 0, A, 0, 64, 8, A, A, T, k, A, A, None)


def swiglu_backward(M, inner):
    return fq.load_library().fp8q_swiglu_backward(A, A, 0, M, inner, A, 0, None)


def quantize(G, K, M=100, rows=False):
    return fq.load_library().fp8q_quantize_act_grouped(A, A, G, M, K, A if rows else 0, A if rows else 0, A, A, None)


def product(G, P, Q, M=100):
    return fq.load_library().fp8q_grouped_gemm_rowscaled(A, A, A, A, A, G, M, P, Q, A, 1, None)


def adamw(*sizes):
    t = (fq._AdamwTensor * len(sizes))(*[fq._AdamwTensor(A, A, A, A, A, A, 0, n) for n in sizes])
    h = fq._AdamwHyper(1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 1, None)
    return fq.load_library().fp8q_adamw(t, len(sizes), 1, 0, ctypes.byref(h), None)


# calls that need 2^32 threads or more
PAST = {"sort, a workgroup per token": lambda: sort(BOUND),
        "sort, FP32 rows of 2048": lambda: sort(BOUND // 2, H=2048, dt=1),
        "sort, long rows": lambda: sort(BOUND // 2, H=16384),
        "sort gradient": lambda: sort_backward(BOUND), "sort gradient, long rows": lambda: sort_backward(BOUND // 4, 7168),
        "combine gradient, four slots per workgroup": lambda: combine_backward(BOUND // 2, 8),
        "SwiGLU gradient": lambda: swiglu_backward(1 << 24, 1 << 11),
        "token tiles of 64 channels": lambda: quantize(1 << 18, 1 << 12), "token tiles of 128": lambda: quantize(1 << 18, 1 << 13, rows=True),
        "weight gradient": lambda: product(1 << 20, 128, 128), "weight gradient, large": lambda: product(1 << 7, 1 << 15, 1 << 15),
        "AdamW, one tensor": lambda: adamw(5, 1 << 35)}


@pytest.mark.parametrize("name", PAST)
def test_past_the_bound(name):
    assert PAST[name]() == E["FP8Q_ERR_SHAPE"]


# the largest ones below
BELOW = {"sort": lambda: sort(BOUND - 1), "sort, long rows, a workgroup per 8192 columns": lambda: sort(BOUND - 1, H=8192),
         "sort gradient": lambda: sort_backward(BOUND - 1), "combine gradient": lambda: combine_backward(BOUND // 2 - 1, 8),
         "SwiGLU gradient": lambda: swiglu_backward((1 << 24) - 1, 1 << 11), "token tiles": lambda: quantize((1 << 18) - 1, 1 << 12),
         "weight gradient": lambda: product((1 << 20) - 1, 128, 128),
         "AdamW, one tensor": lambda: adamw(5, (BOUND - 1) * 2048)}


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would run on fake addresses")
@pytest.mark.parametrize("name", BELOW)
def test_below_the_bound(name):
    assert BELOW[name]() == E["FP8Q_ERR_DEVICE"]
