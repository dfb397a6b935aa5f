"""The norm's gradient and the Newton-Schulz calls by their C entry points, with a workspace of exactly the stated size: nothing
around it is written, and what it held before does not matter."""
import ctypes

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_route_guard import Guarded

pytestmark = pytest.mark.gpu


def rand(shape, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


@pytest.mark.parametrize("T,H", [(0, 64), (1, 8), (5, 1000), (1030, 520), (777, 7168), (9, 8200), (3, 16384)])
def test_norm_gradient(T, H):
    lib, stream = fq.load_library(), torch.cuda.current_stream().cuda_stream
    x, dy, w = rand((T, H), 1), rand((T, H), 2), rand(H, 3)
    _, mean, rstd = fq.fp8q_layer_norm(x, w)
    want = fq.fp8q_layer_norm_backward(dy, x, w, mean, rstd, want_bias=True)
    for fill in (0x5A, 0xFF):  # 0xFF...: NaN
        work, dw, db = Guarded(lib.fp8q_layer_norm_backward_workspace(T, H)), Guarded(4 * H), Guarded(4 * H)
        work.view(torch.uint8, (work.size,)).fill_(fill)
        dx = torch.empty_like(x)
        assert lib.fp8q_layer_norm_backward(dy.data_ptr(), fq.FP8Q_OUT_F32, x.data_ptr(), fq.FP8Q_OUT_F32, w.data_ptr(),
                                            mean.data_ptr(), rstd.data_ptr(), T, H, dx.data_ptr(), fq.FP8Q_OUT_F32, dw.ptr,
                                            db.ptr, work.ptr, stream) == fq.FP8Q_OK
        torch.cuda.synchronize()
        assert work.intact() and dw.intact() and db.intact()
        for a, b in zip((dx, dw.view(torch.float32, (H,)), db.view(torch.float32, (H,))), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 77, 200), (1, 130, 70), (1, 70, 3000), (1, 3000, 70), (1, 256, 7168), (16, 512, 512),
                                   (16, 600, 512), (85, 512, 512), (25, 576, 576), (25, 900, 570), (300, 20, 30)])
def test_newton_schulz(shape):
    """Every size of tile, split and whole sums."""
    lib, stream, (G, P, Q) = fq.load_library(), torch.cuda.current_stream().cuda_stream, shape
    x = rand(shape, 4)
    want = fq.fp8q_orthogonalize(x)
    ns = fq._NewtonSchulz(*fq.NEWTON_SCHULZ, 5)
    for fill in (0x5A, 0xFF):
        work, out = Guarded(lib.fp8q_muon_workspace(G, P, Q)), Guarded(2 * G * P * Q)
        work.view(torch.uint8, (work.size,)).fill_(fill)
        assert lib.fp8q_orthogonalize(x.data_ptr(), fq.FP8Q_OUT_F32, G, P, Q, ctypes.byref(ns), out.ptr, work.ptr, stream) == fq.FP8Q_OK
        torch.cuda.synchronize()
        assert work.intact() and out.intact() and torch.equal(out.view(torch.bfloat16, shape), want)
        work.view(torch.uint8, (work.size,)).fill_(fill)
        p, m = torch.zeros_like(x), torch.zeros_like(x)
        h = fq._MuonHyper(1.0, 0.9, 0.0, 1.0, 1.0, ns, 0, None)
        assert lib.fp8q_muon(p.data_ptr(), x.data_ptr(), fq.FP8Q_OUT_F32, m.data_ptr(), G, P, Q, ctypes.byref(h), 0, work.ptr,
                             stream) == fq.FP8Q_OK
        torch.cuda.synchronize()
        assert work.intact() and torch.equal((-p).bfloat16(), want)
