"""GPU parity of fp8q_adamw.  Every operation of the step is rounded to FP32 by itself, in a
stated order, so numpy's FP32 arithmetic gives the same bits: parameters, FP32 states, E4M3
codes and scales are compared exactly, and the FP32 step with a float64 one within the bound
of its roundings.  Sizes around a chunk of 8, a tile of 128 and a workgroup of 2048, more
tensors than a launch takes, and what lies behind a tensor stays as it was."""
import math

import numpy as np
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from oracle import e4m3
from oracle import quant as oq

from helpers import dev, host

pytestmark = pytest.mark.gpu

F = np.float32
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 0, 127, 128, 129, 2047, 2048, 2049, 5001]


def step_f32(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=1.0):
    """The step in numpy FP32, one rounding per operation."""
    b1, b2 = betas
    decay, size = F(1 - lr * weight_decay), F(lr / (1 - b1 ** step))
    root = F(1 / math.sqrt(1 - b2 ** step))
    g = g.astype(F) * F(grad_scale)
    m = m * F(b1) + g * F(1 - b1)
    v = v * F(b2) + (g * F(1 - b2)) * g
    r = np.sqrt(v)
    return p * decay - (m / (r * root + F(eps))) * size, m, v, r


def tiles(x):
    return np.concatenate([x, np.zeros(-x.size % 128, F)]).reshape(-1, 128)


def to_codes(x, root=False):
    q, s = [], []
    for t in tiles(x):
        a, b = oq.quantize_group(t)
        q.append(np.where((t > 0) & (a == 0), 1, a) if root else a), s.append(b)
    return (np.concatenate(q)[:x.size].astype(np.uint8), np.array(s, F)) if q else (np.zeros(0, np.uint8), np.zeros(0, F))


def of_codes(q, s):
    return (e4m3.decode(q).astype(F) * np.repeat(s, 128)[:q.size]).astype(F)


def bits(a):
    return np.ascontiguousarray(a, F).view(np.uint32)


def draw(sizes, grad, seed, spread=False):
    """Per-tensor numpy inputs; `spread`: magnitudes over many orders and exact zeros."""
    r = np.random.default_rng(seed)
    out = []
    for n in sizes:
        g = r.standard_normal(n) * (10.0 ** r.uniform(-18, 2, n) if spread else 1e-2)
        if spread:
            g[r.random(n) < 0.1] = 0.0
        g = torch.from_numpy(g.astype(F)).to(grad)
        out.append((r.standard_normal(n).astype(F) * F(0.02), g, r.standard_normal(n).astype(F) * F(1e-3),
                    (r.random(n).astype(F) * F(1e-2))))
    return out


def guarded(a, dtype=torch.float32):
    """A device tensor with `a`'s values at the start of a larger buffer of sentinels."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype)
    raw = torch.full((t.numel() + 64,), 77, dtype=dtype, device="cuda")
    raw[:t.numel()] = t.cuda()
    return raw[:t.numel()], raw


def assert_bits(got, ref, what):
    got = host(got)
    bad = np.nonzero(bits(got) != bits(ref))[0]
    assert bad.size == 0, f"{what}: {bad.size} of {ref.size} differ, first at {bad[0]}: {got[bad[0]]!r}, {ref[bad[0]]!r}"


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("copies", [False, True])
def test_f32_states(grad, spread, copies):
    data = draw(SIZES, grad, 1, spread)
    bufs = {k: [guarded(d[i]) for d in data] for i, k in ((0, "p"), (2, "m"), (3, "v"))}
    cp = [guarded(np.zeros(n, F), torch.bfloat16) for n in SIZES] if copies else None
    plan = fq.fp8q_adamw_plan([a for a, _ in bufs["p"]], [d[1].cuda() for d in data], [a for a, _ in bufs["m"]],
                              [a for a, _ in bufs["v"]], copies=[a for a, _ in cp] if copies else None)
    ref = [(d[0], d[2], d[3]) for d in data]
    for step in (1, 2, 3):
        fq.fp8q_adamw(plan, step=step, grad_scale=0.5, **HYPER)
        torch.cuda.synchronize()
        with np.errstate(divide="ignore", invalid="ignore"):
            ref = [step_f32(p, d[1].float().numpy(), m, v, step, grad_scale=0.5, **HYPER)[:3]
                   for d, (p, m, v) in zip(data, ref)]
        for i, r in enumerate(ref):
            for k, x in zip(("p", "m", "v"), r):
                assert_bits(bufs[k][i][0], x, f"step {step}, tensor {i}, {k}")
            if copies:
                assert torch.equal(cp[i][0].cpu(), torch.from_numpy(r[0]).bfloat16()), f"copy {i}"
    for pairs in list(bufs.values()) + ([cp] if copies else []):
        assert all(bool((raw[-64:] == 77).all()) for _, raw in pairs)


def test_f32_step_against_64_bits():
    p, g, m, v = draw([4096], torch.float32, 2)[0]
    t = [dev(x.copy()) for x in (p, g.numpy(), m, v)]
    fq.fp8q_adamw(fq.fp8q_adamw_plan(*[[x] for x in t]), step=7, **HYPER)
    p, g, m, v = (x.astype(np.float64) for x in (p, g.numpy(), m, v))
    b1, b2 = HYPER["betas"]
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    up = HYPER["lr"] * (m2 / (1 - b1 ** 7)) / (np.sqrt(v2 / (1 - b2 ** 7)) + HYPER["eps"])
    p2 = p * (1 - HYPER["lr"] * HYPER["weight_decay"]) - up
    h = 2.0 ** -24
    # m, v: constant, product and sum of two terms, the second of three factors; p: those of m
    # and half of v's, root, product, sum, quotient, step's own rounding; all of size `up`
    big = np.abs(b1 * m) + np.abs((1 - b1) * g)
    assert np.all(np.abs(host(t[2]) - m2) <= 3.1 * h * big)
    assert np.all(np.abs(host(t[3]) - v2) <= 4.1 * h * v2)
    scale = np.maximum(np.abs(up), HYPER["lr"] * big / (1 - b1 ** 7) / (np.sqrt(v2 / (1 - b2 ** 7)) + HYPER["eps"]))
    assert np.all(np.abs(host(t[0]) - p2) <= 12 * h * scale + 3.1 * h * np.abs(p))


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread", [False, True])
def test_e4m3_states(grad, spread):
    data = draw(SIZES, grad, 3, spread)
    bufs = {"p": [guarded(d[0]) for d in data]}
    ref = []
    for name in ("m", "v", "ms", "vs"):
        bufs[name] = []
    for p, _, m, r in data:
        (mq, ms), (vq, vs) = to_codes(m), to_codes(r, True)
        ref.append((p, mq, ms, vq, vs))
        bufs["m"].append(guarded(mq, torch.uint8)), bufs["v"].append(guarded(vq, torch.uint8))
        bufs["ms"].append(guarded(ms)), bufs["vs"].append(guarded(vs))
    plan = fq.fp8q_adamw_plan([a for a, _ in bufs["p"]], [d[1].cuda() for d in data], *[[a for a, _ in bufs[k]] for k in
                                                                                    ("m", "v", "ms", "vs")])
    for step in (1, 2, 3):
        fq.fp8q_adamw(plan, step=step, **HYPER)
        torch.cuda.synchronize()
        new = []
        for d, (p, mq, ms, vq, vs) in zip(data, ref):
            root = of_codes(vq, vs)
            with np.errstate(divide="ignore", invalid="ignore", under="ignore"):
                p, m, _, r = step_f32(p, d[1].float().numpy(), of_codes(mq, ms), root * root, step, **HYPER)
            new.append((p, *to_codes(m), *to_codes(r, True)))
        ref = new
        for i, (p, mq, ms, vq, vs) in enumerate(ref):
            what = f"step {step}, tensor {i}"
            assert_bits(bufs["ms"][i][0], ms, what + " scale of m")
            assert_bits(bufs["vs"][i][0], vs, what + " scale of v")
            assert np.array_equal(host(bufs["m"][i][0]), mq), what + " codes of m"
            assert np.array_equal(host(bufs["v"][i][0]), vq), what + " codes of v"
            assert_bits(bufs["p"][i][0], p, what + " p")
    for pairs in bufs.values():
        assert all(bool((raw[-64:] == 77).all()) for _, raw in pairs)


def test_zero_states_start_a_run():
    """All-zero codes and scales and a zero gradient: nothing but the decay; then a gradient."""
    n = 300
    p = torch.ones(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    st = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(3, device="cuda") for _ in range(2)]
    plan = fq.fp8q_adamw_plan([p], [g], [st[0]], [st[1]], [sc[0]], [sc[1]])
    fq.fp8q_adamw(plan, lr=0.5, weight_decay=0.5, step=1)
    assert bool((p == 0.75).all()) and not any(bool(x.any()) for x in st + sc)
    g.fill_(-2.0)
    fq.fp8q_adamw(plan, lr=0.5, weight_decay=0.0, step=1)
    # the first step moves by lr * g / |g|, up to FP32 rounding (8 operations)
    assert bool(((p - 1.25).abs() <= 8 * 2.0 ** -24).all())


def test_a_small_root_keeps_a_code():
    """One large gradient beside a small one: the small root's code is 1, not 0, so that later
    steps with a zero gradient divide by it, not by eps."""
    g = torch.full((128,), 1e-9, device="cuda")
    g[0] = 1.0
    p, st = torch.zeros(128, device="cuda"), [torch.zeros(128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(1, device="cuda") for _ in range(2)]
    plan = fq.fp8q_adamw_plan([p], [g], [st[0]], [st[1]], [sc[0]], [sc[1]])
    fq.fp8q_adamw(plan, lr=1e-3, step=1)
    assert host(st[1])[1:].tolist() == [1] * 127
    g.zero_()
    for step in range(2, 6):
        fq.fp8q_adamw(plan, lr=1e-3, step=step)
    assert bool(torch.isfinite(p).all()) and float(p.abs().max()) < 5 * 1e-3 * 4


def test_many_tensors_and_scalars():
    """More tensors than a launch takes, shapes of several dimensions, and the device scalars in
    place of lr, step and grad_scale."""
    sizes = [(3 * (i % 17) + 1, 5) for i in range(131)]
    flat = [a * b for a, b in sizes]
    data = draw(flat, torch.float32, 9)
    lists = [[dev(d[i] if i != 1 else d[1].numpy()).reshape(s) for d, s in zip(data, sizes)] for i in range(4)]
    plan = fq.fp8q_adamw_plan(*lists)
    lr, step, b1, b2 = 2e-3, 5, 0.9, 0.95
    sc = torch.tensor([lr, 1 - b1 ** step, 1 - b2 ** step, 0.25], device="cuda")
    fq.fp8q_adamw(plan, lr=123.0, betas=(b1, b2), weight_decay=0.1, step=77, grad_scale=9.0, scalars=sc)
    torch.cuda.synchronize()
    for i, (p, g, m, v) in enumerate(data):
        rp, rm, rv, _ = step_f32(p, g.numpy(), m, v, step, lr, (b1, b2), 1e-8, 0.1, 0.25)
        assert_bits(lists[2][i].reshape(-1), rm, f"m {i}")
        assert_bits(lists[3][i].reshape(-1), rv, f"v {i}")
        # decay, step size and root come from FP32 scalars: a few half-steps more
        assert np.all(np.abs(host(lists[0][i].reshape(-1)) - rp) <= 16 * 2.0 ** -24 * (np.abs(p) + np.abs(rp - p)))
