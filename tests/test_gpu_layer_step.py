"""The calls around the experts together, as a training step makes them: norm, router, sort of the tokens, combine,
and back through the gradients, then Muon on the router's weight and AdamW on the norm's; on streams, from
threads, captured and replayed; the same inputs twice; offsets past 32 bits."""
import math
import threading

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def test_training_step_matches_autograd():
    """One layer whose experts multiply by a factor of their own: y = norm(x), logits = y Wr^T, top-k, rows
    sorted by expert, combined, and the gradients of <out, dy> + loss by x, the norm's weight and bias and Wr,
    against autograd in 64 bits with the chosen experts held.  FP32 throughout: every result is off by
    sums of at most a few hundred terms, taken as 2000 u of its norm."""
    B, S, H, E, k, alpha = 2, 45, 256, 24, 4, 0.05
    T = B * S
    x, dy = rand((T, H), 1), rand((T, H), 2, scale=0.1)
    weight, bias, wr = 1.0 + rand(H, 3, scale=0.1), rand(H, 4, scale=0.1), rand((E, H), 5, scale=0.1)
    gain, steer = 1.0 + rand(E, 6, scale=0.3), rand(E, 7, scale=0.02)
    valid = torch.ones((B, S), dtype=torch.bool, device="cuda")
    valid[1, 30:] = False

    y, mean, rstd = fq.fp8q_layer_norm(x, weight, bias)
    logits = (y @ wr.t()).view(B, S, E)
    ids, w, counts, loss, slope = fq.fp8q_moe_route(logits, k, steer, valid, score="sigmoid", scale=2.0, balance=alpha)
    flat, wf = ids.view(T, k), w.view(T, k)
    xs, offsets, token_row, _ = fq.fp8q_moe_sort(flat, y, 0, E)
    assert torch.equal(offsets[1:] - offsets[:-1], counts.sum(0).int())
    rows = torch.arange(xs.shape[0], device="cuda")
    expert = torch.searchsorted(offsets.long(), rows, right=True).clamp(max=E) - 1
    used = rows < offsets[-1]
    by = torch.where(used, gain[expert.clamp(min=0)], 0.0)[:, None]
    ys = torch.where(used[:, None], xs * by, 0.0)
    out = fq.fp8q_moe_combine(ys, token_row, wf, out_dtype=F32)
    dys, dw = fq.fp8q_moe_combine_backward(dy, ys, token_row, wf)
    dxs = torch.where(used[:, None], dys * by, 0.0)
    dlogits = fq.fp8q_moe_route_backward(logits, ids, w, dw.view(B, S, k), slope, score="sigmoid", scale=2.0).view(T, E)
    dyn = fq.fp8q_moe_sort_backward(dxs, token_row, out_dtype=F32) + dlogits @ wr
    dwr = dlogits.t().contiguous() @ y
    dx, dweight, dbias = fq.fp8q_layer_norm_backward(dyn, x, weight, mean, rstd, want_bias=True)

    d = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    X, W, Bi, R = d(x), d(weight), d(bias), d(wr)
    c = X - X.mean(1, keepdim=True)
    Y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * W + Bi
    s = torch.sigmoid(Y @ R.t())
    at, live = flat.cpu().long(), (flat.cpu() >= 0)
    chosen = torch.where(live, torch.gather(s, 1, at.clamp(min=0)), 0.0)
    wt = 2.0 * chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
    ref = (wt * torch.where(live, gain.double().cpu()[at.clamp(min=0)], 0.0)).sum(1, keepdim=True) * Y
    p = (s / s.sum(1, keepdim=True)).view(B, S, E) * valid.cpu()[..., None]
    L = (slope.double().cpu() * p.sum(1)).sum()
    ((ref * dy.double().cpu()).sum() + L).backward()

    def near(a, b, what):
        off = (a.double().cpu() - b.detach()).norm() / b.detach().norm()
        assert off <= 2000 * U, (what, off.item())

    near(out, ref, "out")
    near(loss, L.reshape(1), "loss")
    near(dx, X.grad, "dx")
    near(dweight, W.grad, "dweight")
    near(dbias, Bi.grad, "dbias")
    near(dwr, R.grad, "dwr")

    # the optimizers: Muon for the router's weight, AdamW for the norm's
    before, m = wr.clone(), torch.zeros_like(wr)
    fq.fp8q_muon(wr, dwr, m, lr=0.01, scale=1.0)
    o = ((before - wr) / 0.01).double()
    s = torch.linalg.svdvals(o.cpu())
    assert (s > 0.3).all() and (s < 1.3).all() and torch.equal(m, dwr)
    plan = fq.fp8q_adamw_plan([weight, bias], [dweight, dbias], *[[torch.zeros_like(weight) for _ in range(2)] for _ in range(2)])
    old = weight.clone()
    fq.fp8q_adamw(plan, lr=1e-3)
    # the first step moves every value by lr, less where the gradient is as small as eps
    assert ((old - weight).abs() <= 1.001e-3).all() and ((old - weight).sign() == dweight.sign())[dweight.abs() > 1e-6].all()


class Step:
    """The new calls on fixed buffers of inputs."""

    def __init__(self, seed):
        self.x, self.dy = rand((200, 520), seed, BF16), rand((200, 520), seed + 1, BF16)
        self.weight, self.bias = 1.0 + rand(520, seed + 2, scale=0.1), rand(520, seed + 3)
        self.logits, self.steer = rand((4, 50, 70), seed + 4), rand(70, seed + 5, scale=0.1)
        self.valid = torch.rand((4, 50), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) < 0.8
        self.dw, self.grad = rand((4, 50, 6), seed + 6), rand((3, 140, 300), seed + 7, BF16)
        self.long = rand((130, 4200), seed + 8)  # a split product
        self.param, self.momentum = rand((3, 140, 300), seed + 9), rand((3, 140, 300), seed + 10)

    def inputs(self):
        return [self.x, self.dy, self.weight, self.bias, self.logits, self.steer, self.valid, self.dw, self.grad, self.long,
                self.param, self.momentum]

    def __call__(self, stream=None):
        kw = {} if stream is None else {"stream": stream}
        y, mean, rstd = fq.fp8q_layer_norm(self.x, self.weight, self.bias, **kw)
        back = fq.fp8q_layer_norm_backward(self.dy, self.x, self.weight, mean, rstd, want_bias=True, **kw)
        routed = fq.fp8q_moe_route(self.logits, 6, self.steer, self.valid, balance=0.1, **kw)
        one = fq.fp8q_moe_route(self.logits[0, :20], 6, self.steer, balance=0.1, **kw)
        dz = fq.fp8q_moe_route_backward(self.logits, routed[0], routed[1], self.dw, routed[4], **kw)
        o, q = fq.fp8q_orthogonalize(self.grad, **kw), fq.fp8q_orthogonalize(self.long, **kw)
        fq.fp8q_muon(self.param, self.grad, self.momentum, lr=0.1, **kw)
        return [y, mean, rstd, *back, *routed, *one, dz, o, q, self.param, self.momentum]


def same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


def test_the_same_inputs_twice():
    same([t.clone() for t in Step(1)()], Step(1)())


def test_on_another_stream():
    want = [t.clone() for t in Step(2)()]
    torch.cuda.synchronize()
    s = Step(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s(side)
    side.synchronize()
    same(got, want)
    s = Step(2)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s()
    side.synchronize()
    same(got, want)
    s = Step(2)
    side.wait_stream(torch.cuda.current_stream())
    got = s(side.cuda_stream)
    side.synchronize()
    same(got, want)


def test_two_streams_and_threads_at_once():
    want = [[t.clone() for t in Step(10 * i)()] for i in range(3)]
    torch.cuda.synchronize()
    got, errors = [None] * 3, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(3):
                    got[i] = Step(10 * i)()
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for g, w in zip(got, want):
        same(g, w)


def test_captured_and_replayed():
    """Two graphs of the same calls share a memory pool and run in turn; every replay equals an eager run."""
    s = Step(20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            outs.append(s())
        graphs.append(g)
    for rep in range(4):
        fresh = Step(30 + rep)
        for mine, theirs in zip(s.inputs(), fresh.inputs()):
            mine.copy_(theirs)
        want = [t.clone() for t in fresh()]
        _ = fq.fp8q_orthogonalize(rand((64, 64), rep))  # other work in between
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        same(outs[rep % 2], want)


def test_captured_step_with_a_device_learning_rate():
    p, g, m = rand((40, 90), 1), rand((40, 90), 2), torch.zeros((40, 90), device="cuda")
    lr = torch.full((1,), 0.5, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.fp8q_muon(p.clone(), g, m.clone(), lr=1.0, device_lr=lr)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fp8q_muon(p, g, m, lr=1.0, weight_decay=0.1, device_lr=lr)
    p2, m2 = p.clone(), m.clone()
    for rate in (0.5, 0.125, 0.03):
        lr.fill_(rate)
        graph.replay()
        fq.fp8q_muon(p2, g, m2, lr=rate, weight_decay=0.1)
        torch.cuda.synchronize()
        assert torch.equal(p, p2) and torch.equal(m, m2)


def test_offsets_past_32_bits():
    """The last rows, tokens and matrices of tensors with more than 2^31 elements are those of the same alone."""
    T, H = 270_000, 8192
    x = torch.zeros((T, H), device="cuda", dtype=BF16)
    x[-3:] = rand((3, H), 1, BF16)
    w = torch.ones(H, device="cuda")
    y, mean, rstd = fq.fp8q_layer_norm(x, w)
    y3, mean3, rstd3 = fq.fp8q_layer_norm(x[-3:].contiguous(), w)
    assert torch.equal(y[-3:], y3) and torch.equal(mean[-3:], mean3) and not y[:-3].any()
    dx, dw, _ = fq.fp8q_layer_norm_backward(x, x, w, mean, rstd)
    dx3, dw3, _ = fq.fp8q_layer_norm_backward(x[-3:].contiguous(), x[-3:].contiguous(), w, mean3, rstd3)
    assert torch.equal(dx[-3:], dx3) and (dw - dw3).norm() <= 100 * U * dw3.norm()
    del x, y, dx
    z = torch.zeros((2, 4_200_000, 256), device="cuda", dtype=BF16)
    z[1, -5:] = rand((5, 256), 2, BF16)
    ids, wt, counts, loss, slope = fq.fp8q_moe_route(z, 2, balance=0.1)
    few = fq.fp8q_moe_route(z[1, -5:].contiguous(), 2)
    assert torch.equal(ids[1, -5:], few[0]) and torch.equal(wt[1, -5:], few[1]) and counts.sum().item() == 4 * 4_200_000
    dz = fq.fp8q_moe_route_backward(z, ids, wt, torch.ones_like(wt), torch.zeros_like(slope))
    dz3 = fq.fp8q_moe_route_backward(z[1, -5:].contiguous(), few[0], few[1], torch.ones_like(few[1]), slope[1] * 0)
    assert torch.equal(dz[1, -5:], dz3)
    del z, dz, ids, wt
    G, P, Q = 132, 4096, 4096
    x = torch.zeros((G, P, Q), device="cuda", dtype=BF16)
    x[-1] = rand((P, Q), 3, BF16)
    out = fq.fp8q_orthogonalize(x, steps=1)
    alone = fq.fp8q_orthogonalize(x[-1].contiguous(), steps=1)
    assert not out[:-1].any()
    # other tiles, the same sums: BF16 results differ where a rounding to FP16 in between does
    assert (out[-1].double() - alone.double()).norm() <= 1e-3 * alone.double().norm()
