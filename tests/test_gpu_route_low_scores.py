"""Sigmoid scores of tokens whose logits are all far below zero: the shares p = s / sum s, and with them the balance
loss and the gradient, stay those of the definition where every score is below FP32's range.

Tolerances are those of test_gpu_route.py: a share is formed relative to e^min(top, 0) with one exponential of a
difference of at most R, one reciprocal and a sum, as a normalized weight is, and carries no more roundings than it."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from test_gpu_route import U, by_autograd, check_forward, spread_of

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def low(S, E, dtype, level, seed):
    """Logits around `level`, with a spread of a few units."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (level - 3.0 * torch.rand((2, S, E), device="cuda", generator=g)).to(dtype)


def check(z, k, bias, valid, normalize):
    ids, w, counts, loss, slope = check_forward(z, k, bias, valid, "sigmoid", normalize, scale=1.5, balance=0.3)
    assert torch.isfinite(loss).all() and loss.item() > 0
    dw = torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8))
    dloss = torch.full((1,), 1.75, device="cuda")
    live = z.float() if valid is None else torch.where(valid[..., None], z.float(), 0.0)
    for odt in (F32, BF16):
        dz = fq.fp8q_moe_route_backward(z, ids, w, dw, slope, dloss, score="sigmoid", normalize=normalize, scale=1.5, out_dtype=odt)
        rz, size = by_autograd(z, ids.cpu().long(), "sigmoid", normalize, 1.5, slope.double().cpu(), dw.double().cpu(), 1.75)
        tol = (100 + 4 * spread_of(live)) * U * size + 1e-37
        tol = tol + torch.finfo(odt).eps / 2 * (rz.abs() + tol)
        assert ((dz.double().cpu() - rz).abs() <= tol).all()


@pytest.mark.parametrize("level", [-0.5, -10.0, -17.0, -60.0, -85.0, -87.0, -90.0, -103.0, -200.0, -600.0])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (60, 3), (128, 8), (256, 8), (300, 5), (1024, 8)])
@pytest.mark.parametrize("normalize", [True, False])
def test_all_scores_low(E, k, level, normalize):
    """BF16 and FP32, with and without a bias that steers the choice."""
    for dtype, with_bias in ((F32, True), (F32, False), (BF16, True)):
        z = low(9, E, dtype, level, E + k)
        b = 0.1 * torch.randn(E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) if with_bias else None
        check(z, k, b, None, normalize)


@pytest.mark.parametrize("E,k", [(64, 4), (256, 8), (600, 8)])
@pytest.mark.parametrize("fill", [-90.0, -200.0, -1e9, torch.finfo(F32).min])
def test_low_tokens_beside_others(E, k, fill):
    """Tokens filled with one large negative number between ordinary ones, some of their experts masked, others
    padded with NaN: shares of 1 / E each, or of 1 / (experts left)."""
    g = torch.Generator(device="cuda").manual_seed(E)
    z = torch.randn((2, 37, E), device="cuda", generator=g)
    v = torch.rand((2, 37), device="cuda", generator=g) < 0.8
    v[0, 5] = v[1, 36] = v[0, 9] = True
    z[0, 5] = z[1, 36] = z[0, 9] = fill
    z[0, 9, ::2] = -torch.inf
    z[~v] = torch.nan
    b = 0.1 * torch.randn(E, device="cuda", generator=g)
    ids, w, counts, loss, slope = fq.fp8q_moe_route(z, k, b, v, score="sigmoid", balance=0.3)
    assert torch.isfinite(loss).all() and torch.isfinite(slope).all()
    # the loss: sums of shares in 64 bits; the three rows' are equal over their experts
    s = torch.sigmoid(torch.where(v[..., None], z, 0.0).double())
    flat = torch.ones(E, device="cuda", dtype=torch.float64)
    s[0, 5], s[1, 36], s[0, 9] = flat, flat, flat * (z[0, 9] > -torch.inf)
    p = torch.where(v[..., None], s / s.sum(-1, keepdim=True), 0.0)
    want = (slope.double() * p.sum(1)).sum().item()
    assert abs(loss.item() - want) <= 200 * U * want
    dw = torch.randn(w.shape, device="cuda", generator=g)
    dz = fq.fp8q_moe_route_backward(z, ids, w, dw, slope, score="sigmoid")
    assert torch.isfinite(dz).all() and not dz[~v].any() and not dz[0, 9, ::2].any()
    # a row of equal logits: s is 0 beside 1, p is 1 / n, w = 1 / k; the bound is that of a gradient's terms with R = 0,
    # each sum taken by its largest term
    for at, n in (((0, 5), E), ((1, 36), E), ((0, 9), E // 2)):
        gs, d, i = slope[at[0]].double(), dw[at].double(), ids[at].long()
        keep = (z[at] > -torch.inf).double()
        mean = (gs * keep).sum() / n
        one = keep * (gs - mean) / n
        one.scatter_add_(0, i, (d - d.mean()) / k)
        size = (gs.abs() + gs.abs().max()) / n
        size.scatter_add_(0, i, (d.abs() + d.abs().max()) / k)
        assert ((dz[at].double() - one).abs() <= 100 * U * size).all(), at


@pytest.mark.parametrize("low_at", [[0], [3], [1, 2], []])
def test_neighbours_do_not_change_a_token(low_at):
    """A token's results are the same bits beside tokens with low scores in its wave and without them."""
    g = torch.Generator(device="cuda").manual_seed(2)
    z = torch.randn((4, 100), device="cuda", generator=g)
    z[:, 0] = 0.5
    y = z.clone()
    for t in low_at:
        y[t] -= 300.0
    kept = [t for t in range(4) if t not in low_at]
    slope = 0.01 * torch.rand(100, device="cuda", generator=g)
    outs = []
    for x in (z, y):
        ids, w, *_ = fq.fp8q_moe_route(x, 5, score="sigmoid")
        outs.append((ids, w, fq.fp8q_moe_route_backward(x, ids, w, torch.ones_like(w), slope, score="sigmoid")))
    for a, c in zip(*outs):
        assert torch.equal(a[kept], c[kept])


def test_low_scores_captured_and_replayed():
    z = low(20, 256, F32, -90.0, 3)
    z[0, 1::2] += 90.0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.fp8q_moe_route(z, 8, score="sigmoid", balance=0.1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fq.fp8q_moe_route(z, 8, score="sigmoid", balance=0.1)
        dz = fq.fp8q_moe_route_backward(z, out[0], out[1], torch.ones_like(out[1]), out[4], score="sigmoid")
    for level in (0.0, -50.0, 40.0, -400.0):
        z.copy_(low(20, 256, F32, -90.0 + level, 4))
        want = [t.clone() for t in fq.fp8q_moe_route(z, 8, score="sigmoid", balance=0.1)]
        want.append(fq.fp8q_moe_route_backward(z, want[0], want[1], torch.ones_like(want[1]), want[4], score="sigmoid"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip((*out, dz), want):
            assert torch.isfinite(a).all() and torch.equal(a, c)
