"""Values that are not finite stay with the token, row or matrix they came in: the results beside them are the same bits."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu
BAD = [torch.nan, torch.inf]


def rand(shape, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(16, 2), (60, 8), (256, 8), (300, 64), (1024, 5)])
def test_router(E, k, score, bad):
    """Tokens that count with such logits, some experts or all: ids below E, the others' ids, weights, counts and gradient
    kept, and the other sequence's slope."""
    z, b = rand((2, 40, E), E), 0.1 * rand(E, 1)
    odd = torch.zeros((2, 40), dtype=torch.bool, device="cuda")
    odd[0, 3] = odd[0, 17] = odd[0, 39] = True
    y = z.clone()
    y[0, 3], y[0, 17, 1], y[0, 39, ::2] = bad, bad, bad
    for bias in (b, None):
        clean = fq.fp8q_moe_route(z, k, bias, score=score, balance=0.3)
        got = fq.fp8q_moe_route(y, k, bias, score=score, balance=0.3)
        assert ((got[0] >= -1) & (got[0] < E)).all()
        for i in (0, 1):
            assert torch.equal(got[i][~odd], clean[i][~odd])
        assert torch.equal(got[2][1], clean[2][1]) and torch.equal(got[4][1], clean[4][1])
        dw, slope = rand(clean[1].shape, 2), rand((2, E), 3)
        want = fq.fp8q_moe_route_backward(z, clean[0], clean[1], dw, slope, score=score)
        dz = fq.fp8q_moe_route_backward(y, got[0], got[1], dw, slope, score=score)
        assert torch.equal(dz[~odd], want[~odd])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T,H", [(7, 64), (600, 1000), (1100, 8), (9, 8200)])
def test_norm(T, H, bad):
    x, dy, w, b = rand((T, H), 1), rand((T, H), 2), rand(H, 3), rand(H, 4)
    kept = torch.arange(T, device="cuda") != T // 2
    y = x.clone()
    y[T // 2, H // 2] = bad
    for center in (True, False):
        clean, got = (fq.fp8q_layer_norm(t, w, b, center=center) for t in (x, y))
        assert torch.equal(got[0][kept], clean[0][kept]) and torch.equal(got[2][kept], clean[2][kept])
        want = fq.fp8q_layer_norm_backward(dy, x, w, clean[1], clean[2])[0]
        assert torch.equal(fq.fp8q_layer_norm_backward(dy, y, w, got[1], got[2])[0][kept], want[kept])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("shape", [(3, 20, 30), (3, 130, 200), (3, 200, 130), (3, 70, 3000), (16, 512, 512), (16, 600, 512), (85, 600, 512),
                                   (40, 500, 900), (25, 900, 570)])
def test_newton_schulz(shape, bad):
    x = rand(shape, 5)
    kept = torch.arange(shape[0], device="cuda") != 1
    y = x.clone()
    y[1, -1, -1] = bad
    assert torch.equal(fq.fp8q_orthogonalize(y)[kept], fq.fp8q_orthogonalize(x)[kept])
    outs = []
    for g in (x, y):
        p, m = torch.ones_like(x), torch.zeros_like(x)
        fq.fp8q_muon(p, g, m, lr=0.1)
        outs.append((p[kept], m[kept]))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
