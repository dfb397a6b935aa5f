"""Layer norm and RMS norm and their gradients against their formulas in 64 bits.

Tolerances, with u = 2^-24 (half a step of FP32): a sum over a row is a tree of at most 8 or 16 terms of a
thread, 6 levels of a wave and 16 waves, so it is off by at most 40 u of the sum of magnitudes; a sum over
rows by ceil(T / 256) + 4 rows of a workgroup, 16 workgroups of a slice and 16 slices.  Every other step
rounds once, and a result of another type by half a step of it."""
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def inputs(T, H, dtype, seed, shift=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), device="cuda", generator=g) + shift * torch.randn((1, H), device="cuda", generator=g)
    w = 1.0 + 0.2 * torch.randn(H, device="cuda", generator=g)
    b = 0.3 * torch.randn(H, device="cuda", generator=g)
    return x.to(dtype), w, b


def half_step(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs() + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def reference(x, w, b, eps, center):
    x, w = x.double(), w.double()
    mean = x.mean(1, keepdim=True) if center else torch.zeros((x.shape[0], 1), dtype=torch.float64, device=x.device)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    return d * rstd * w + (b.double() if b is not None else 0), mean, rstd, d * rstd


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("xdt,ydt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (777, 1000), (64, 7168), (1100, 520), (5, 8192), (3, 8200), (2, 16384)])
def test_forward(T, H, xdt, ydt, center):
    x, w, b = inputs(T, H, xdt, T + H)
    y, mean, rstd = fq.fp8q_layer_norm(x, w, b if center else None, eps=1e-5, center=center, out_dtype=ydt)
    ry, rm, rr, h = reference(x, w, b if center else None, 1e-5, center)
    a = x.double().abs().mean(1, keepdim=True)
    dm = 41 * U * a if center else 0 * a
    assert y.dtype == ydt and (mean is None) == (not center)
    if center:
        assert ((mean.double()[:, None] - rm).abs() <= dm).all()
    # the squares' mean: off by 40 u, and by twice the error of the mean against values of size 1 / rstd
    dr = rr * (25 * U + (dm * rr) ** 2 + 2 * U)
    assert ((rstd.double()[:, None] - rr).abs() <= dr).all()
    tol = w.double().abs() * (dm * rr * (1 + h.abs()) + h.abs() * 32 * U) + 2 * U * (ry.abs() + b.double().abs())
    tol = tol + half_step(ry.abs() + tol, ydt)
    assert ((y.double() - ry).abs() <= tol).all()


def test_far_mean_and_equal_rows():
    """A mean far above the spread keeps the squares of x - mean; a row of equal values gives the bias."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 4096.0 + torch.randint(-8, 9, (9, 512), device="cuda", generator=g).float()
    x[4] = 7.0
    w, b = torch.ones(512, device="cuda"), torch.full((512,), 0.25, device="cuda")
    y, mean, rstd = fq.fp8q_layer_norm(x, w, b)
    ry, _, rr, h = reference(x, w, b, 1e-5, True)
    # mean off by 41 u 4096 = 0.01 at the most, against a spread of 5
    tol = 41 * U * 4104 * rr * (1 + h.abs()) + 64 * U * (1 + h.abs())
    keep = torch.arange(9, device="cuda") != 4
    assert ((y.double() - ry).abs() <= tol)[keep].all()
    assert (y[4] == 0.25).all() and mean[4] == 7.0 and rstd[4] == (1 / torch.sqrt(torch.tensor(1e-5))).item()


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("ddt,xdt,odt", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16), (F32, BF16, F32)])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (777, 1000), (1030, 520), (64, 7168), (5, 8192), (9, 8200), (2, 16384)])
def test_backward(T, H, ddt, xdt, odt, center):
    x, w, b = inputs(T, H, xdt, T + H + 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    dy = torch.randn((T, H), device="cuda", generator=g).to(ddt)
    _, mean, rstd = fq.fp8q_layer_norm(x, w, b, center=center)
    dx, dw, db = fq.fp8q_layer_norm_backward(dy, x, w, mean, rstd, want_bias=center, out_dtype=odt)
    assert dx.dtype == odt and (db is None) == (not center)
    # the formulas with the statistics as given
    xd, d, r = x.double(), dy.double(), rstd.double()[:, None]
    h = (xd - mean.double()[:, None] if center else xd) * r
    gw = d * w.double()
    s, t = (gw * h).mean(1, keepdim=True), gw.mean(1, keepdim=True) * center
    rx = r * (gw - t - h * s)
    ds, dt = 44 * U * (gw * h).abs().mean(1, keepdim=True), 42 * U * gw.abs().mean(1, keepdim=True) * center
    tol = r * (h.abs() * ds + dt + 6 * U * (gw.abs() + t.abs() + (h * s).abs()))
    assert ((dx.double() - rx).abs() <= tol + half_step(rx.abs() + tol, odt)).all()
    n = -(-T // 256) + 4 + 32
    assert ((dw.double() - (d * h).sum(0)).abs() <= (n + 4) * U * (d * h).abs().sum(0)).all()
    if center:
        assert ((db.double() - d.sum(0)).abs() <= n * U * d.abs().sum(0)).all()


@pytest.mark.parametrize("center", [True, False])
def test_backward_against_differences(center):
    """Along random directions, <dx, u> + <dweight, v> + <dbias, q> is the derivative of <dy, y>.  Central
    differences with step e in 64 bits are off by their second-order term, about e^2; the gradients by the
    bound of test_backward, here summed as 200 u of the magnitudes."""
    T, H, e = 7, 40, 1e-4
    x, w, b = inputs(T, H, F32, 11)
    g = torch.Generator(device="cuda").manual_seed(12)
    dy, u = (torch.randn((T, H), device="cuda", generator=g) for _ in range(2))
    v, q = (torch.randn(H, device="cuda", generator=g) for _ in range(2))
    _, mean, rstd = fq.fp8q_layer_norm(x, w, b, center=center)
    dx, dw, db = fq.fp8q_layer_norm_backward(dy, x, w, mean, rstd, want_bias=True)

    def value(k):
        y = reference(x.double() + k * u.double(), w.double() + k * v.double(), b.double() + k * q.double(), 1e-5, center)[0]
        return (y * dy.double()).sum()

    slope = ((value(e) - value(-e)) / (2 * e)).item()
    terms = [(a.double() * c.double()) for a, c in ((dx, u), (dw, v), (db, q))]
    got, size = sum(t.sum().item() for t in terms), sum(t.abs().sum().item() for t in terms)
    assert abs(got - slope) <= size * (200 * U + 100 * e * e)


def test_no_tokens():
    w = torch.ones(64, device="cuda")
    x = torch.zeros((0, 64), device="cuda", dtype=BF16)
    y, mean, rstd = fq.fp8q_layer_norm(x, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = fq.fp8q_layer_norm_backward(x, x, w, mean, rstd, want_bias=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_outputs_stay_in_their_buffers():
    T, H = 37, 1000
    x, w, b = inputs(T, H, BF16, 4)
    raw = torch.full(((T + 2) * H,), 7.0, device="cuda", dtype=BF16)
    y, mean, rstd = fq.fp8q_layer_norm(x, w, b, y=raw[H:-H].view(T, H))
    assert (raw[:H] == 7).all() and (raw[-H:] == 7).all()
    want, _, _ = fq.fp8q_layer_norm(x, w, b)
    assert torch.equal(y, want)
    fq.fp8q_layer_norm_backward(x, x, w, mean, rstd, dx=raw[H:-H].view(T, H))
    assert (raw[:H] == 7).all() and (raw[-H:] == 7).all()


def test_refusals():
    x, w, b = inputs(4, 64, BF16, 1)
    m = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="weight"):
        fq.fp8q_layer_norm(x, w[:32])
    with pytest.raises(ValueError, match="contiguous"):
        fq.fp8q_layer_norm(x.t().contiguous().t(), w)
    with pytest.raises(ValueError, match="weight"):
        fq.fp8q_layer_norm(x, w.bfloat16())
    with pytest.raises(ValueError, match="dy must be"):
        fq.fp8q_layer_norm_backward(x[:, :32].contiguous(), x, w, m, m)
    with pytest.raises(ValueError, match="rstd"):
        fq.fp8q_layer_norm_backward(x, x, w, None, m[:3])
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_layer_norm(x, w, eps=-1.0)
    wide = torch.zeros((1, 16392), device="cuda")
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_layer_norm(wide, torch.zeros(16392, device="cuda"))
