"""The router over as many sequences as a grid takes: ids and weights are those of the same tokens as one sequence, counts,
slope and loss those of the definition.  Tolerances are those of test_gpu_route.py."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_route import U, scores, spread_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,S,E,k", [(65535, 1, 16, 2), (65535, 3, 60, 8), (4000, 9, 300, 5), (65535, 0, 8, 2)])
def test_many_sequences(B, S, E, k, score):
    g = torch.Generator(device="cuda").manual_seed(B + S)
    z = torch.randn((B, S, E), device="cuda", generator=g)
    bias = 0.1 * torch.randn(E, device="cuda", generator=g)
    ids, w, counts, loss, slope = fq.fp8q_moe_route(z, k, bias, score=score, balance=0.3)
    one = fq.fp8q_moe_route(z.view(-1, E), k, bias, score=score)
    assert torch.equal(ids.view(-1, k), one[0]) and torch.equal(w.view(-1, k), one[1]) and torch.equal(counts.sum(0).int(), one[2].view(E))
    by_hand = torch.zeros((B, E), device="cuda", dtype=torch.int32)
    by_hand.scatter_add_(1, ids.view(B, -1).long(), torch.ones_like(ids.view(B, -1)))
    assert torch.equal(counts, by_hand)
    want = 0.3 / B * E * counts.double() / max(S * S * k, 1)
    assert ((slope.double() - want).abs() <= 1.01 * U * want + 1e-45).all()
    total = (slope.double() * scores(z.double(), score)[1].sum(1)).sum().item()
    assert abs(loss.item() - total) <= (120 + S / 256 + 2 * spread_of(z)) * U * total if S else loss.item() == 0
    dz = fq.fp8q_moe_route_backward(z, ids, w, torch.ones_like(w), slope, score=score)
    for b in (0, B // 2, B - 1):  # each alone, with its own slope
        alone = fq.fp8q_moe_route_backward(z[b], ids[b], w[b], torch.ones_like(w[b]), slope[b], score=score)
        assert torch.equal(dz[b], alone)
