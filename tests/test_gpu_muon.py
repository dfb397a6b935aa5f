"""Orthogonalized matrices and Muon steps against the polynomial of the singular values in 64 bits.

Tolerances: the roundings to FP16 that the kernels make by design are made on a model of the iteration in
64 bits (`model`); its distance from the exact result, measured for each input, is what these roundings cost.
The kernels differ from the model by FP32 sums, which move some roundings to the other neighbour, so they are
allowed twice that distance, and 1e-6 of the norm.  The result's rounding to BF16 is off by 2^-8 of a value at
the most, and by 2^-8 / sqrt(3) in the mean over many."""
import math

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ABC = fq.NEWTON_SCHULZ


def half(t):
    """Rounded to FP16 at the kernels' scale."""
    return (t * 4096.0).half().double() / 4096.0


def low(t):
    """What is left of X behind FP16, rounded to E4M3 at the kernels' scale."""
    return (t * (4096.0 * 256)).float().clamp(-448, 448).to(torch.float8_e4m3fn).double() / (4096.0 * 256)


def exact(x, steps=5, abc=ABC):
    """From the singular values, which the iteration changes alone."""
    u, s, v = torch.linalg.svd(x.double().cpu(), full_matrices=False)
    n = s.norm(dim=-1, keepdim=True)
    s = torch.where(n > 0, s / n, 0.0)
    for _ in range(steps):
        s = s * (abc[0] + abc[1] * s ** 2 + abc[2] * s ** 4)
    return (u * s[..., None, :]) @ v


def by_products(x, steps=5, abc=ABC, rounded=False):
    """The iteration in 64 bits, with the kernels' roundings to FP16 if asked for."""
    x = x.double()
    if x.shape[-2] > x.shape[-1]:
        return by_products(x.transpose(-1, -2), steps, abc, rounded).transpose(-1, -2)
    n = x.flatten(-2).norm(dim=-1)[..., None, None]
    x = torch.where(n > 0, x / n, 0.0)
    eye = torch.eye(x.shape[-2], dtype=torch.float64, device=x.device)
    r = half if rounded else (lambda t: t)
    for _ in range(steps):
        hi = r(x)
        lo = low(x - hi) if rounded else x - hi
        a = hi @ hi.transpose(-1, -2).contiguous()
        d = a * eye
        o = r(a - d)
        c = abc[0] * eye + abc[1] * (o + d) + abc[2] * ((o + d) @ (o + d))
        dc = c.diagonal(dim1=-2, dim2=-1)[..., None]
        dh = r(dc)
        turn = torch.where(dh.abs() * 4096 >= 2.0 ** -13, dc / dh, 1.0)
        x = turn * ((r(c - dc * eye) + dh * eye) @ hi) + dc * lo
    return x


def allowed(x, steps=5, abc=ABC):
    """(exact result, its norm per matrix, what the roundings in between may cost)."""
    e = by_products(x, steps, abc)
    m = by_products(x, steps, abc, rounded=True)
    norm = e.flatten(-2).norm(dim=-1)
    return e, norm, 2 * (m - e).flatten(-2).norm(dim=-1) + 1e-6 * norm


def matrices(shape, kind, dtype=F32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    x = n(*shape)
    if kind == "strong":  # a few directions over a floor of noise
        r = min(5, *shape[-2:])
        x = 0.02 * x + torch.matmul(n(*shape[:-1], r), n(*shape[:-2], r, shape[-1])) / math.sqrt(r)
    return x.to(dtype)


SHAPES = [(1, 1), (1, 7), (7, 1), (5, 3), (8, 8), (64, 64), (65, 63), (100, 130), (128, 128), (129, 257), (300, 1000),
          (1000, 300), (513, 512), (3, 77, 200), (4, 200, 77), (2, 256, 640),
          (128, 7168), (7168, 200), (2, 70, 3000)]


@pytest.mark.parametrize("kind", ["normal", "strong"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(shape, kind):
    for dtype in (F32, BF16):
        x = matrices(shape, kind, dtype, sum(shape))
        before = x.clone()
        out = fq.fp8q_orthogonalize(x)
        assert out.dtype == BF16 and out.shape == x.shape and torch.equal(x, before)
        e, norm, inside = allowed(x)
        off = (out.double() - e).flatten(-2).norm(dim=-1)
        rounding = norm * 2.0 ** -8 * (0.6 if x[..., 0, 0].numel() * shape[-1] * shape[-2] > 2000 else 1.0)
        assert (off <= torch.sqrt(inside ** 2 + rounding ** 2)).all(), (off / norm).max()
        assert ((e.cpu() - exact(x)).abs() <= 1e-9 * (1 + norm.max().item())).all()


@pytest.mark.parametrize("shape", [(85, 512, 512), (25, 576, 576), (40, 500, 900), (25, 900, 570)])
def test_larger_tiles(shape):
    """Batches that fill the CUs with tiles of 192 or 256."""
    x = matrices(shape, "strong", BF16, 3)
    e, norm, inside = allowed(x)
    off = (fq.fp8q_orthogonalize(x).double() - e).flatten(-2).norm(dim=-1)
    assert (off <= torch.sqrt(inside ** 2 + (norm * 0.6 * 2.0 ** -8) ** 2)).all()


@pytest.mark.parametrize("shape", [(16, 512, 512), (16, 600, 512), (12, 600, 500), (32, 1000, 500), (85, 600, 512)])
def test_tiles_of_128_and_tall_ones_of_256(shape):
    """Batches of a few hundred tiles of 128, and tall matrices' tiles of 256."""
    x = matrices(shape, "strong", BF16, 4)
    e, norm, inside = allowed(x)
    off = (fq.fp8q_orthogonalize(x).double() - e).flatten(-2).norm(dim=-1)
    assert (off <= torch.sqrt(inside ** 2 + (norm * 0.6 * 2.0 ** -8) ** 2)).all()


@pytest.mark.parametrize("steps,abc", [(1, ABC), (2, ABC), (8, ABC), (12, (1.875, -1.25, 0.375)), (3, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(steps, abc):
    for shape in ((90, 150), (150, 90)):
        x = matrices(shape, "normal", F32, 5)
        e, norm, inside = allowed(x, steps, abc)
        off = (fq.fp8q_orthogonalize(x, steps=steps, coefficients=abc).double() - e).norm()
        assert off <= torch.sqrt(inside ** 2 + (norm * 0.6 * 2.0 ** -8) ** 2)


def test_scale_of_the_input_does_not_matter():
    x = matrices((60, 90), "normal")
    want = fq.fp8q_orthogonalize(x)
    for k in (2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 2.0 ** 120):  # squares far outside FP32
        assert torch.equal(fq.fp8q_orthogonalize(x * k), want)


def test_zeros_stay_zeros_beside_others():
    x = matrices((3, 50, 70), "normal")
    x[1] = 0
    out = fq.fp8q_orthogonalize(x)
    assert not out[1].any() and torch.equal(out[0], fq.fp8q_orthogonalize(x[0].contiguous()))
    assert torch.equal(out[2], fq.fp8q_orthogonalize(x[2].contiguous()))


def test_nothing_to_do():
    for shape in ((0, 5), (5, 0), (0, 4, 4), (3, 0, 8)):
        assert fq.fp8q_orthogonalize(torch.zeros(shape, device="cuda")).shape == shape


def step(p, g, m, lr, beta, nesterov, decay, scale, grad_scale=1.0):
    """New (param, momentum), the update and what its roundings may cost, in 64 bits."""
    g = g.double() * grad_scale
    m = beta * m.double() + g
    u = g + beta * m if nesterov else m
    e, _, inside = allowed(u)
    return p.double() * (1 - lr * decay) - lr * scale * e, m, e, inside


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(9, 14), (128, 384), (300, 77), (3, 130, 100), (25, 576, 576)])
def test_muon(shape, nesterov):
    lr, beta, decay, scale = 0.02, 0.9, 0.1, 1.5
    for dtype, copy in ((BF16, True), (F32, False)):
        p, m = matrices(shape, "normal", F32, 1), 0.5 * matrices(shape, "strong", F32, 2)
        g = matrices(shape, "strong", dtype, 3)
        rp, rm, e, inside = step(p, g, m, lr, beta, nesterov, decay, scale, 0.5)
        c = torch.zeros(shape, device="cuda", dtype=BF16) if copy else None
        fq.fp8q_muon(p, g, m, lr=lr, beta=beta, nesterov=nesterov, weight_decay=decay, scale=scale, grad_scale=0.5, copy=c)
        # momentum: two roundings of FP32, beta's own among three of the first term
        assert ((m.double() - rm).abs() <= 2.0 ** -24 * (3 * rm.abs() + 4 * (g.double().abs()))).all()
        off = (p.double() - rp).flatten(-2).norm(dim=-1)
        size = 2.0 ** -24 * (4 * rp.flatten(-2).norm(dim=-1) + 8 * lr * scale * e.flatten(-2).norm(dim=-1))
        assert (off <= lr * scale * inside + size).all()
        if copy:
            assert torch.equal(c, p.bfloat16())


@pytest.mark.parametrize("shape", [(2, 70, 320), (3, 321, 128), (70, 3000), (200, 260), (260, 200), (16, 512, 512), (16, 600, 512),
                                   (12, 600, 500), (32, 1000, 512), (32, 1000, 500), (40, 500, 900), (85, 512, 512)])
def test_muon_over_tiles(shape):
    """Tiles of every size, whole and cut by the matrix's right and lower edge, beside the next matrix's rows."""
    lr, beta, decay, scale = 0.02, 0.9, 0.1, 1.5
    n = math.prod(shape)
    p, m = matrices(shape, "normal", F32, 1), 0.5 * matrices(shape, "strong", F32, 2)
    g = matrices(shape, "strong", BF16, 3)
    rp, _, e, inside = step(p, g, m, lr, beta, True, decay, scale, 1.0)
    raws = [torch.full((n + 128,), 7.0, device="cuda", dtype=dtype) for dtype in (F32, BF16)]
    q, c = (raw[64:64 + n].view(shape) for raw in raws)
    q.copy_(p)
    fq.fp8q_muon(q, g, m, lr=lr, beta=beta, weight_decay=decay, scale=scale, copy=c)
    off = (q.double() - rp).flatten(-2).norm(dim=-1)
    size = 2.0 ** -24 * (4 * rp.flatten(-2).norm(dim=-1) + 8 * lr * scale * e.flatten(-2).norm(dim=-1))
    assert (off <= lr * scale * inside + size).all()
    # an element's error is a part of its matrix's
    assert ((q.double() - rp).abs().flatten(-2).amax(dim=-1) <= lr * scale * inside + size).all()
    assert torch.equal(c, q.bfloat16())
    for raw in raws:
        assert (raw[:64] == 7).all() and (raw[64 + n:] == 7).all()


def test_muon_default_scale_and_device_lr():
    shape = (40, 100)
    p0, m0, g = matrices(shape, "normal", F32, 1), matrices(shape, "normal", F32, 2), matrices(shape, "normal", F32, 3)
    runs = []
    for kw in (dict(lr=0.01), dict(lr=0.01, scale=0.2 * 10.0), dict(lr=5.0, device_lr=torch.full((1,), 0.01, device="cuda"))):
        p, m = p0.clone(), m0.clone()
        fq.fp8q_muon(p, g, m, weight_decay=0.1, **kw)
        runs.append((p, m))
    for p, m in runs[1:]:
        assert torch.equal(p, runs[0][0]) and torch.equal(m, runs[0][1])


def test_outputs_stay_in_their_buffers():
    for shape in ((33, 50), (50, 33), (128, 128)):
        n = shape[0] * shape[1]
        def inside(dtype, fill):
            raw = torch.full((n + 128,), fill, device="cuda", dtype=dtype)
            return raw, raw[64:64 + n].view(shape)
        raws = []
        raw, out = inside(BF16, 7.0)
        raws.append(raw)
        x = matrices(shape, "normal")
        fq.fp8q_orthogonalize(x, out=out)
        assert torch.equal(out, fq.fp8q_orthogonalize(x))
        views = {}
        for name, dtype in (("param", F32), ("momentum", F32), ("copy", BF16)):
            raw, views[name] = inside(dtype, 7.0)
            raws.append(raw)
        fq.fp8q_muon(views["param"], x, views["momentum"], lr=0.1, copy=views["copy"])
        for raw in raws:
            assert (raw[:64] == 7).all() and (raw[64 + n:] == 7).all() and not (raw[64:64 + n] == 7).all()


def test_refusals():
    x = matrices((8, 16), "normal")
    with pytest.raises(ValueError, match="contiguous"):
        fq.fp8q_orthogonalize(x.t())
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        fq.fp8q_orthogonalize(x.half())
    with pytest.raises(ValueError, match=r"\[P, Q\]"):
        fq.fp8q_orthogonalize(x[0].contiguous())
    with pytest.raises(ValueError, match="out"):
        fq.fp8q_orthogonalize(x, out=torch.zeros((8, 16), device="cuda"))
    for bad in (dict(steps=0), dict(steps=101), dict(coefficients=(math.nan, 1, 1))):
        with pytest.raises(fq.Fp8qError):
            fq.fp8q_orthogonalize(x, **bad)
    p, m = x.clone(), x.clone()
    for bad in (dict(lr=math.inf), dict(lr=0.1, beta=1.0), dict(lr=0.1, beta=-0.5), dict(lr=0.1, weight_decay=math.nan)):
        with pytest.raises(fq.Fp8qError):
            fq.fp8q_muon(p, x, m, **bad)
    with pytest.raises(ValueError, match="share memory"):
        fq.fp8q_muon(p, x, p, lr=0.1)
    with pytest.raises(ValueError, match="param"):
        fq.fp8q_muon(p.bfloat16(), x, m, lr=0.1)
    with pytest.raises(ValueError, match="momentum"):
        fq.fp8q_muon(p, x, m[:4], lr=0.1)
    with pytest.raises(ValueError, match="copy"):
        fq.fp8q_muon(p, x, m, lr=0.1, copy=m)
