"""The router's C entry points with a workspace of exactly the stated size and with outputs of their own size:
nothing around them is written, sequences without tokens among the batches."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu
GUARD = 32768  # bytes on either side


class Guarded:
    """`size` bytes between guard bytes."""

    def __init__(self, size):
        self.size = size
        self.raw = torch.full((size + 2 * GUARD,), 0x5A, device="cuda", dtype=torch.uint8)
        self.ptr = self.raw.data_ptr() + GUARD

    def view(self, dtype, shape):
        return self.raw[GUARD:GUARD + self.size].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:GUARD] == 0x5A).all()) and bool((self.raw[GUARD + self.size:] == 0x5A).all())


@pytest.mark.parametrize("score", [fq.FP8Q_SCORE_SOFTMAX, fq.FP8Q_SCORE_SIGMOID])
@pytest.mark.parametrize("B,S,E,k", [(8, 0, 256, 8), (2, 0, 1024, 64), (3, 0, 16, 2), (1, 0, 64, 4), (300, 0, 257, 3), (1, 1, 256, 8),
                                     (1, 32, 60, 3), (1, 33, 60, 3), (8, 1, 1, 1), (4, 70, 1024, 64), (5, 9, 257, 7),
                                     (2, 8300, 64, 4)])
def test_nothing_around_is_written(B, S, E, k, score):
    lib, stream = fq.load_library(), torch.cuda.current_stream().cuda_stream
    g = torch.Generator(device="cuda").manual_seed(B + S + E)
    z = torch.randn((B, S, E), device="cuda", generator=g)
    bias = 0.1 * torch.randn(E, device="cuda", generator=g)
    work = Guarded(lib.fp8q_moe_route_workspace(B, S, E))
    ids, w, dz = Guarded(4 * B * S * k), Guarded(4 * B * S * k), Guarded(4 * B * S * E)
    counts, slope, loss = Guarded(4 * B * E), Guarded(4 * B * E), Guarded(4)
    assert lib.fp8q_moe_route(z.data_ptr(), fq.FP8Q_OUT_F32, B, S, E, k, bias.data_ptr(), 0, score, 1, 1.0, 0.1, ids.ptr, w.ptr,
                              counts.ptr, loss.ptr, slope.ptr, work.ptr, stream) == fq.FP8Q_OK
    dw = torch.randn((B, S, k), device="cuda", generator=g)
    assert lib.fp8q_moe_route_backward(z.data_ptr(), fq.FP8Q_OUT_F32, B, S, E, k, ids.ptr, w.ptr, dw.data_ptr(), slope.ptr, 0,
                                       score, 1, 1.0, dz.ptr, fq.FP8Q_OUT_F32, stream) == fq.FP8Q_OK
    torch.cuda.synchronize()
    for name, t in dict(work=work, ids=ids, w=w, counts=counts, slope=slope, loss=loss, dz=dz).items():
        assert t.intact(), name
    assert (counts.view(torch.int32, (B, E)).sum(1) == S * k).all()
    chosen = ids.view(torch.int32, (B, S, k))
    assert ((chosen >= 0) & (chosen < E)).all()
    assert torch.isfinite(dz.view(torch.float32, (B, S, E))).all() and torch.isfinite(w.view(torch.float32, (B, S, k))).all()
    if S == 0:
        assert not slope.view(torch.float32, (B, E)).any() and loss.view(torch.float32, (1,)).item() == 0
