"""The router against its definition in 64 bits: ids, counts exactly, weights, slope, loss and the gradient
within bounds.

Tolerances, with u = 2^-24: exp is off by 2 u of itself and its argument, a difference of logits of size
R at the most, by u R; a sum over experts is a tree of at most 16 + 6 levels, over a sequence's tokens of
at most S / 256 + 64 more.  A weight is a score over a sum of at most 64: (40 + 2 R) u of itself.  A loss is a sum
of positive terms: (120 + S / 256 + 2 R) u of itself.  A gradient's terms p g, p sum(p g), w dw and w sum(w dw)
carry at most (100 + 4 R) u of their magnitudes."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def make(B, S, E, dtype, seed, bias, padded):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (1.5 * torch.randn((B, S, E), device="cuda", generator=g) + torch.randn((1, 1, E), device="cuda", generator=g)).to(dtype)
    b = 0.1 * torch.randn(E, device="cuda", generator=g) if bias else None
    v = torch.rand((B, S), device="cuda", generator=g) < 0.7 if padded else None
    return z, b, v


def scores(z, score):
    """Scores and shares of the experts, float64 torch on the CPU."""
    s = torch.softmax(z, -1) if score == "softmax" else torch.sigmoid(z)
    return s, s / s.sum(-1, keepdim=True)


def reference(z, k, bias, valid, score, normalize, scale, balance):
    """ids, weights, counts, loss, slope from the definition, with rows that count."""
    z = z.double().cpu()
    B, S, E = z.shape
    live = torch.isfinite(z).any(-1) & (torch.ones((B, S), dtype=torch.bool) if valid is None else valid.cpu())
    z = torch.where(live[..., None], z, torch.zeros(()).double())
    s, p = scores(z, score)
    rank = (z if bias is None else s + bias.double().cpu()).masked_fill(z == -torch.inf, -torch.inf)
    ids = torch.from_numpy(np.argsort(-rank.numpy(), axis=-1, kind="stable")[..., :k].copy())
    gone = torch.gather(z, -1, ids) == -torch.inf
    ids = torch.where(gone | ~live[..., None], -1, ids)
    w = torch.where(ids >= 0, torch.gather(s, -1, ids.clamp(min=0)), 0.0)
    if normalize:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    w = w * scale
    counts = (ids.reshape(B, -1, 1) == torch.arange(E)).sum(1) if S else torch.zeros((B, E), dtype=torch.long)
    n = live.sum(1, keepdim=True).double()
    slope = balance / B * E * counts.double() / (n * counts.sum(1, keepdim=True)).clamp(min=1)
    loss = (slope * torch.where(live[..., None], p, 0.0).sum(1)).sum()
    return ids, w, counts, loss, slope, live


def spread_of(z):
    d = z.double()
    d = d[torch.isfinite(d)]
    return (d.max() - d.min()).item() if d.numel() else 0.0


def check_forward(z, k, bias, valid, score, normalize, scale=2.5, balance=0.01):
    ids, w, counts, loss, slope = fq.fp8q_moe_route(z, k, bias, valid, score=score, normalize=normalize, scale=scale, balance=balance)
    ri, rw, rc, rl, rs, live = reference(z, k, bias, valid, score, normalize, scale, balance)
    assert torch.equal(ids.cpu().long(), ri)
    R = spread_of(torch.where(live.to(z.device)[..., None], z, torch.zeros((), device=z.device, dtype=z.dtype)))
    assert ((w.cpu().double() - rw).abs() <= (40 + 2 * R) * U * rw + 1e-37).all()
    assert torch.equal(counts.cpu().long(), rc)
    assert ((slope.cpu().double() - rs).abs() <= 1.01 * U * rs + 1e-45).all()
    assert abs(loss.item() - rl.item()) <= (120 + z.shape[1] / 256 + 2 * R) * U * rl.item() + 1e-45
    return ids, w, counts, loss, slope


EXPERTS = [(1, 1), (4, 4), (5, 2), (37, 3), (60, 8), (64, 64), (65, 1), (100, 7), (128, 20), (200, 33), (256, 8), (257, 5),
           (600, 64), (1023, 8), (1024, 17)]


@pytest.mark.parametrize("E,k", EXPERTS)
@pytest.mark.parametrize("score,normalize,bias", [("softmax", True, False), ("softmax", False, True), ("sigmoid", True, True),
                                                  ("sigmoid", False, False)])
def test_forward_experts(E, k, score, normalize, bias):
    for dtype, B, S in ((F32, 2, 33), (BF16, 1, 7)):
        z, b, v = make(B, S, E, dtype, E + k, bias, True)
        check_forward(z, k, b, v, score, normalize)


@pytest.mark.parametrize("B,S", [(1, 1), (1, 32), (1, 33), (5, 1), (3, 700), (1, 9000), (2, 8193)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_forward_tokens(B, S, score):
    z, b, v = make(B, S, 64, F32, S, True, True)
    check_forward(z, 4, b, v, score, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", ["none", "zero", "few"])
def test_ties_go_to_the_lowest_index(score, bias):
    """Logits of few values: many experts tie, also behind the k-th."""
    g = torch.Generator(device="cuda").manual_seed(9)
    z = torch.randint(-2, 3, (3, 50, 96), device="cuda", generator=g).to(BF16)
    b = None if bias == "none" else torch.zeros(96, device="cuda")
    if bias == "few":
        b[::3] = 0.125
    check_forward(z, 16, b, None, score, True)


def test_near_ties_are_ranked_in_64_bits():
    """Scores + biases closer than FP32 tells apart: expert e's bias makes up for its logit but for 1e-9 e."""
    E = 40
    z = torch.linspace(-1.5, 1.5, E).repeat(1, 9, 1).cuda()
    s = torch.sigmoid(z[0, 0].double().cpu())
    order = torch.randperm(E, generator=torch.Generator().manual_seed(1)).double()
    b = (0.9 - s + 3e-8 * order).float().cuda()
    check_forward(z.contiguous(), 12, b, None, "sigmoid", True)
    s = torch.softmax(z[0, 0].double().cpu(), -1)
    b = (0.1 - s + 4e-9 * order).float().cuda()
    check_forward(z.contiguous(), 12, b, None, "softmax", False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(64, 8), (250, 60), (256, 8), (1024, 64)])
def test_many_equal_scores(score, E, k):
    """All experts alike but for a few: more experts than FP32 tells apart, up to all of them, beside tokens
    without ties in the same wave."""
    g = torch.Generator(device="cuda").manual_seed(E)
    z = torch.randn((2, 37, E), device="cuda", generator=g)
    z[:, ::3] = 0.25
    z[:, ::6, ::50] = 0.5
    z[0, 9] = -torch.inf
    z[0, 9, 3::7] = -1.0
    z[1, 4, : E // 2] = 1.0 + 1e-7 * torch.randint(0, 3, (E // 2,), device="cuda", generator=g)
    b = torch.zeros(E, device="cuda")
    check_forward(z, k, b, None, score, True)
    b[5:40] = 3e-8 * torch.randint(0, 4, (35,), device="cuda", generator=g)
    check_forward(z, k, b, None, score, False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_tokens_and_sequences(score):
    """-inf experts, rows without any, padded rows of NaN and of inf, a sequence without a token."""
    z, b, v = make(4, 21, 48, F32, 3, True, True)
    z[:, :, ::4] = -torch.inf
    z[0, 3, 2:] = -torch.inf          # fewer experts than slots
    z[0, 5] = -torch.inf              # none
    v[0, 3] = v[0, 5] = True
    v[2] = False
    z[~v] = torch.nan
    z[1, ~v[1]] = torch.inf
    ids, w, counts, loss, slope = check_forward(z, 6, b, v, score, True)
    assert torch.isfinite(w).all() and torch.isfinite(loss).all() and torch.isfinite(slope).all()
    assert (ids[2] == -1).all() and not counts[2].any() and not slope[2].any()
    dw = torch.randn(w.shape, device="cuda")
    dw[ids < 0] = torch.nan
    dz = fq.fp8q_moe_route_backward(z, ids, w, dw, slope, score=score)
    assert torch.isfinite(dz).all() and not dz[~v].any() and not dz[0, 5].any()
    assert not dz[..., ::4].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [-torch.inf, torch.finfo(F32).min, -1e9, -30.0])
def test_experts_masked_by_their_bias(score, mask):
    """Half of the experts with a bias that keeps them from being chosen, and more slots than the others fill."""
    z, b, v = make(2, 70, 200, F32, 11, True, True)
    b[1::2] = mask
    ids, w, *_ = check_forward(z, 8, b, v, score, True)
    assert not (ids[v] & 1).any()
    b[4:] = mask
    if mask > -torch.inf:  # those are taken in their order all the same
        check_forward(z, 8, b, v, score, True)
        return
    b[1] = 0.0
    ids, w, counts, loss, slope = fq.fp8q_moe_route(z, 8, b, v, score=score, balance=0.01)
    assert (ids[v][:, 3:] == -1).all() and not w[v][:, 3:].any() and (ids[~v] == -1).all()
    assert (ids[v][:, :3].sort(-1).values == torch.tensor([0, 1, 2], device="cuda")).all()
    assert torch.isfinite(w).all() and torch.isfinite(loss).all() and (counts[:, :3] == v.sum(1, keepdim=True)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    """Normalized weights of chosen experts whose scores vanish together in FP32 stay finite."""
    z = -200.0 - torch.arange(24.0, device="cuda").repeat(1, 5, 1)
    z[:, :, 20:] = 60.0
    b = torch.zeros(24, device="cuda")
    b[20:] = -10.0                    # the large ones are not chosen
    ids, w, *_ = check_forward(z.contiguous(), 4, b, None, score, True)
    assert (ids < 20).all() and (w.sum(-1) - 2.5).abs().max() < 1e-5


def test_no_tokens_and_no_loss():
    z = torch.zeros((3, 0, 16), device="cuda")
    ids, w, counts, loss, slope = fq.fp8q_moe_route(z, 2, balance=0.1)
    assert ids.shape == (3, 0, 2) and not counts.any() and loss.item() == 0 and not slope.any()
    z, _, _ = make(2, 40, 16, F32, 1, False, False)
    _, _, counts, loss, slope = fq.fp8q_moe_route(z, 2)
    assert counts.sum().item() == 2 * 40 * 2 and loss.item() == 0 and not slope.any()


def test_two_dimensional_logits():
    z, b, v = make(1, 77, 60, F32, 2, True, True)
    one = fq.fp8q_moe_route(z, 3, b, v, balance=0.1)
    two = fq.fp8q_moe_route(z[0], 3, b, v[0], balance=0.1)
    for x, y in zip(one, two):
        assert torch.equal(x.reshape(-1), y.reshape(-1)) and (y.dim() == x.dim() - 1 or x.numel() == 1)
    dw = torch.randn_like(one[1])
    a = fq.fp8q_moe_route_backward(z, one[0], one[1], dw, one[4])
    c = fq.fp8q_moe_route_backward(z[0], two[0], two[1], dw[0], two[4])
    assert torch.equal(a[0], c)


def by_autograd(z, ids, score, normalize, scale, slope, dw, dloss):
    """d (sum dw w + dloss loss) / d logits in 64 bits, and a bound of the terms' magnitudes."""
    z = z.double().cpu()
    live = ids[..., :1] >= 0
    z = torch.where(live, z, 0.0).requires_grad_()
    s, p = scores(z, score)
    chosen = torch.where(ids >= 0, torch.gather(s, -1, ids.clamp(min=0)), 0.0)
    w = scale * (chosen / chosen.sum(-1, keepdim=True).clamp(min=1e-300) if normalize else chosen)
    dw = torch.where(ids >= 0, dw, 0.0)
    g = slope[:, None, :] * dloss
    value = (w * dw).sum() + torch.where(live, g * p, 0.0).sum()
    value.backward()
    with torch.no_grad():
        a = (w * dw).abs()
        size = torch.where(live, p * (g.abs() + (p * g).abs().sum(-1, keepdim=True) + a.sum(-1, keepdim=True)), 0.0)
        size = size.scatter_add(-1, ids.clamp(min=0), torch.where(ids >= 0, a + w * a.sum(-1, keepdim=True) / scale, 0.0))
    return z.grad, size


@pytest.mark.parametrize("E,k", EXPERTS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_backward(E, k, score, normalize):
    for dtype, odt, B, S in ((F32, F32, 2, 33), (BF16, BF16, 1, 70), (BF16, F32, 1, 3)):
        z, b, v = make(B, S, E, dtype, E + k, True, True)
        scale = 1.5
        ids, w, _, _, slope = fq.fp8q_moe_route(z, k, b, v, score=score, normalize=normalize, scale=scale, balance=0.3)
        dw = torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8))
        dloss = torch.full((1,), 1.75, device="cuda")
        dz = fq.fp8q_moe_route_backward(z, ids, w, dw, slope, dloss, score=score, normalize=normalize, scale=scale, out_dtype=odt)
        rz, size = by_autograd(z, ids.cpu().long(), score, normalize, scale, slope.double().cpu(), dw.double().cpu(), 1.75)
        tol = (100 + 4 * spread_of(z)) * U * size + 1e-37
        tol = tol + torch.finfo(odt).eps / 2 * (rz.abs() + tol)
        assert dz.dtype == odt and ((dz.double().cpu() - rz).abs() <= tol).all(), (dtype, odt)


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_backward_against_differences(score, normalize):
    """Along a random direction of the logits, in 64 bits and with the chosen experts and counts held."""
    z, b, v = make(2, 9, 24, F32, 5, True, True)
    ids, w, counts, _, slope = fq.fp8q_moe_route(z, 4, b, v, score=score, normalize=normalize, balance=0.3)
    dw, u = torch.randn_like(w), torch.randn_like(z)
    dz = fq.fp8q_moe_route_backward(z, ids, w, dw, slope, score=score, normalize=normalize)
    at, live, e = ids.cpu().long(), ids.cpu()[..., :1] >= 0, 1e-4

    def value(x):
        s, p = scores(x, score)
        c = torch.gather(s, -1, at.clamp(min=0))
        c = c / c.sum(-1, keepdim=True) if normalize else c
        return (torch.where(live, c * dw.double().cpu(), 0.0).sum() + torch.where(live, slope.double().cpu()[:, None] * p, 0.0).sum()).item()

    zd, ud = z.double().cpu(), u.double().cpu()
    slope_ = (value(zd + e * ud) - value(zd - e * ud)) / (2 * e)
    terms = dz.double().cpu() * ud
    assert abs(terms.sum().item() - slope_) <= terms.abs().sum().item() * 300 * U + 100 * e * e * terms.abs().sum().item()


def test_ids_out_of_range_are_skipped():
    """Ids that are not the router's: below 0 or past the last expert they count for nothing, twice the same add up."""
    z, _, _ = make(1, 6, 16, F32, 4, False, False)
    ids, w, _, _, slope = fq.fp8q_moe_route(z, 3, score="sigmoid", normalize=False)
    dw = torch.ones_like(w)
    odd = ids.clone()
    odd[..., 1] = 99
    odd[..., 2] = -5
    one = ids.clone()
    one[..., 1:] = -1
    a = fq.fp8q_moe_route_backward(z, odd, w, dw, slope, score="sigmoid", normalize=False)
    c = fq.fp8q_moe_route_backward(z, one, w, dw, slope, score="sigmoid", normalize=False)
    assert torch.equal(a, c)


def test_refusals():
    z, b, v = make(2, 5, 16, F32, 1, True, True)
    for bad in (dict(k=0), dict(k=17), dict(k=65)):
        with pytest.raises(ValueError, match="k must"):
            fq.fp8q_moe_route(z, **bad)
    with pytest.raises(ValueError, match="score"):
        fq.fp8q_moe_route(z, 2, score="tanh")
    with pytest.raises(ValueError, match="valid"):
        fq.fp8q_moe_route(z, 2, valid=v[:1])
    with pytest.raises(ValueError, match="valid"):
        fq.fp8q_moe_route(z, 2, valid=v.to(torch.uint8))
    with pytest.raises(ValueError, match="bias"):
        fq.fp8q_moe_route(z, 2, bias=b[:8])
    with pytest.raises(ValueError, match="contiguous"):
        fq.fp8q_moe_route(z.transpose(0, 1), 2)
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_moe_route(torch.zeros((2, 1025), device="cuda"), 2)
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_moe_route(z, 2, scale=0.0)
    ids, w, _, _, slope = fq.fp8q_moe_route(z, 2)
    with pytest.raises(ValueError, match="dw"):
        fq.fp8q_moe_route_backward(z, ids, w, w[..., :1], slope)
    with pytest.raises(ValueError, match="dloss"):
        fq.fp8q_moe_route_backward(z, ids, w, w, slope, torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="slope"):
        fq.fp8q_moe_route_backward(z, ids, w, w, slope[:1])
