"""Tokens that no expert is left for, by their logits and the bias together: they count for nothing, in the loss and in its
gradient alike.  Tolerances are those of test_gpu_route.py."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_route import U, by_autograd, scores, spread_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,S,E,k", [(1, 5, 8, 2), (2, 33, 60, 3), (1, 20, 256, 8), (3, 70, 300, 5)])
def test_tokens_without_an_expert(B, S, E, k, score):
    """Every third token has logits for the experts below E / 2 alone, which the bias masks."""
    g = torch.Generator(device="cuda").manual_seed(E)
    z = torch.randn((B, S, E), device="cuda", generator=g)
    z[:, ::3, E // 2:] = -torch.inf
    bias = 0.1 * torch.randn(E, device="cuda", generator=g)
    bias[:E // 2] = -torch.inf
    lone = torch.zeros((B, S), dtype=torch.bool, device="cuda")
    lone[:, ::3] = True
    ids, w, counts, loss, slope = fq.fp8q_moe_route(z, k, bias, score=score, balance=0.3)
    assert (ids[lone] == -1).all() and not w[lone].any() and (ids[~lone] >= E // 2).all()
    # the other tokens are routed, counted and averaged as if these were not there
    rest = z[~lone].view(B, -1, E)
    n = rest.shape[1]
    r_ids, r_w, r_counts, r_loss, r_slope = fq.fp8q_moe_route(rest, k, bias, score=score, balance=0.3)
    assert torch.equal(ids[~lone], r_ids.view(-1, k)) and torch.equal(w[~lone], r_w.view(-1, k)) and torch.equal(counts, r_counts)
    assert torch.equal(slope, r_slope)
    p = scores(rest.double().cpu(), score)[1]
    want = (r_slope.double().cpu() * p.sum(1)).sum().item()
    assert abs(loss.item() - want) <= (120 + S / 256 + 2 * spread_of(z)) * U * want
    assert abs(slope.sum().item() / (0.3 / n * E) - 1) <= 1e-5  # balance / B * E / n for each sequence
    dw = torch.randn(w.shape, device="cuda", generator=g)
    dz = fq.fp8q_moe_route_backward(z, ids, w, dw, slope, score=score)
    assert not dz[lone].any()
    rz, size = by_autograd(rest, r_ids.cpu().long(), score, True, 1.0, r_slope.double().cpu(), dw[~lone].view(B, -1, k).double().cpu(), 1.0)
    tol = (100 + 4 * spread_of(z)) * U * size + 1e-37
    assert ((dz[~lone].view(B, -1, E).double().cpu() - rz).abs() <= tol * (1 + 2 * U)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_no_token_with_an_expert(score):
    z = torch.randn((2, 40, 16), device="cuda")
    ids, w, counts, loss, slope = fq.fp8q_moe_route(z, 2, torch.full((16,), -torch.inf, device="cuda"), score=score, balance=0.3)
    assert (ids == -1).all() and not w.any() and not counts.any() and loss.item() == 0 and not slope.any()
