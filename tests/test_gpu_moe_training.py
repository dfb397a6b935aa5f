"""One MoE layer's training step, put together from the entry points as a program would: sort,
quantize, grouped GEMMs and SwiGLU forward, the gradients of the combine, the activations, the
tokens and both expert weights, and AdamW on the weights.

* against the layer without quantization in float64 (autograd), within the errors of the E4M3
  roundings on the way;
* captured into a HIP graph and replayed with new routings, tokens and step scalars, every
  replay equal to an eager run of the same calls, bit for bit;
* on a side stream given as an argument, and from two host threads at once, equal to the run
  on the default stream;
* outputs between guard bytes, and sizes whose offsets pass 31 bits."""
import threading

import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

from test_gpu_guard import Guarded, assert_intact, p, run

pytestmark = pytest.mark.gpu

T, K_TOP, EXPERTS, E0, LOCAL, H, I = 300, 4, 32, 4, 8, 512, 256
CAP = T * K_TOP


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def inputs(seed):
    g = gen(seed)
    score = torch.rand((T, EXPERTS), device="cuda", generator=g)
    score[:, E0 + 2] = 0.0                                            # an expert without tokens
    top = torch.topk(score, K_TOP, dim=1)
    return {"ids": top.indices.to(torch.int32), "gate": top.values / top.values.sum(1, keepdim=True),
            "x": torch.randn((T, H), device="cuda", generator=g).bfloat16(),
            "dy": (torch.randn((T, H), device="cuda", generator=g) * 1e-2).bfloat16()}


def parameters(seed, e4m3=True):
    g = gen(seed)
    up = torch.randn((LOCAL, 2 * I, H), device="cuda", generator=g) * H ** -0.5
    down = torch.randn((LOCAL, H, I), device="cuda", generator=g) * I ** -0.5
    par = {"p": [up, down], "copy": [up.bfloat16(), down.bfloat16()], "g": [torch.empty_like(up), torch.empty_like(down)]}
    state = torch.uint8 if e4m3 else torch.float32
    par["m"], par["v"] = ([torch.zeros(t.shape, dtype=state, device="cuda") for t in par["p"]] for _ in range(2))
    if e4m3:
        par["ms"], par["vs"] = ([torch.zeros(t.numel() // 128, device="cuda") for t in par["p"]] for _ in range(2))
    par["plan"] = fq.fp8q_adamw_plan(par["p"], par["g"], par["m"], par["v"], par.get("ms"), par.get("vs"), par["copy"])
    return par


def step(d, par, scalars=None, stream=None, update=True):
    """One training step of the layer; returns what it computes."""
    kw = {"stream": stream}
    xs, off, tr, _ = fq.fp8q_moe_sort(d["ids"], d["x"], E0, LOCAL, **kw)
    xq, sx, xt, sxt = fq.fp8q_quantize_act_grouped(xs, off, **kw)
    uq, su, uqt, sut = fq.fp8q_quantize_w_128x128_t(par["copy"][0], **kw)
    dq, sd, dqt, sdt = fq.fp8q_quantize_w_128x128_t(par["copy"][1], **kw)
    gu = fq.fp8q_grouped_gemm_blockscaled(xq, sx, uq, su, off, **kw)
    hq, sh = fq.fp8q_swiglu_quantize_act_1x128(gu, **kw)
    ys = fq.fp8q_grouped_gemm_blockscaled(hq, sh, dq, sd, off, **kw)
    y = fq.fp8q_moe_combine(ys, tr, d["gate"], **kw)
    dys, dgate = fq.fp8q_moe_combine_backward(d["dy"], ys, tr, d["gate"], **kw)
    dyq, sdy, dyt, sdyt = fq.fp8q_quantize_act_grouped(dys, off, **kw)
    dh = fq.fp8q_grouped_gemm_blockscaled(dyq, sdy, dqt, sdt, off, **kw)
    dgu, h = fq.fp8q_swiglu_backward(gu, dh, want_h=True, **kw)
    guq, sgu, gut, sgut = fq.fp8q_quantize_act_grouped(dgu, off, **kw)
    _, _, ht, sht = fq.fp8q_quantize_act_grouped(h, off, rows=False, **kw)
    dxs = fq.fp8q_grouped_gemm_blockscaled(guq, sgu, uqt, sut, off, **kw)
    dx = fq.fp8q_moe_sort_backward(dxs, tr, out_dtype=torch.float32, **kw)
    fq.fp8q_grouped_gemm_rowscaled(gut, sgut, xt, sxt, off, CAP, out=par["g"][0], **kw)
    fq.fp8q_grouped_gemm_rowscaled(dyt, sdyt, ht, sht, off, CAP, out=par["g"][1], **kw)
    if update:
        fq.fp8q_adamw(par["plan"], lr=1e-3, weight_decay=0.1, step=1, scalars=scalars, **kw)
    return {"y": y, "dgate": dgate, "dx": dx, "dup": par["g"][0], "ddown": par["g"][1], "off": off, "tr": tr}


def state(par):
    return [t for k in ("p", "copy", "m", "v", "ms", "vs") for t in par.get(k, [])]


def same(a, b, what):
    for k in a:
        assert torch.equal(a[k], b[k]), f"{what}: {k}"


def kept(out):
    return {k: v.clone() for k, v in out.items()}


def test_step_against_64_bits():
    d, par = inputs(1), parameters(2)
    out = step(d, par, update=False)
    torch.cuda.synchronize()
    x = d["x"].double().requires_grad_()
    gate = d["gate"].double().requires_grad_()
    up, down = (w.double().requires_grad_() for w in par["copy"])
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(LOCAL):
        t, s = torch.nonzero(d["ids"] == E0 + e, as_tuple=True)
        gu = x[t] @ up[e].t()
        g, u = gu[:, :I], gu[:, I:]
        y = y.index_add(0, t, gate[t, s, None] * ((g * torch.sigmoid(g) * u) @ down[e].t()))
    y.backward(d["dy"].double())
    # E4M3 rounds by at most 2^-4 relative, so by 2^-4 / sqrt(3) rms; a result is a product of sums
    # with at most six rounded factors behind it, whose errors add in the square, and SwiGLU, a
    # product of two of them, doubles what comes in: sqrt(6) * 2 * 0.036 = 0.18 of the norm.
    for k, ref in (("y", y), ("dgate", gate.grad), ("dx", x.grad), ("dup", up.grad), ("ddown", down.grad)):
        ref = ref.detach()
        rel = float((out[k].double() - ref).norm() / ref.norm())
        print(f"[{k}] error {rel:.4f} of the norm", flush=True)
        assert rel < 0.18, k
    assert bool((out["dup"][2] == 0).all()) and bool((out["ddown"][2] == 0).all())


def test_adamw_moves_both_experts_weights():
    d, par = inputs(1), parameters(2)
    before = [t.clone() for t in par["p"]]
    out = step(d, par)
    torch.cuda.synchronize()
    for w, b, g, c in zip(par["p"], before, (out["dup"], out["ddown"]), par["copy"]):
        # the first step moves every weight with a gradient by lr against its sign, beside the decay
        moved = w - b * (1 - 1e-4)
        here = g.abs() > 1e-6
        assert bool(((moved + 1e-3 * g.sign()).abs()[here] < 1e-3 * 0.02).all())
        assert torch.equal(c, w.bfloat16())
        assert torch.equal(w[2], (b * torch.tensor(1 - 1e-4, device="cuda"))[2])   # no tokens: decay alone


def test_graph_replays_match_eager():
    d, par, eager = inputs(3), parameters(4), parameters(4)
    b1, b2 = 0.9, 0.95
    scalars = torch.tensor([1e-3, 1 - b1, 1 - b2, 1.0], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(d, parameters(4), scalars)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(d, par, scalars)
    for rep in range(4):
        for k, v in inputs(10 + rep).items():
            d[k].copy_(v)
        scalars.copy_(torch.tensor([1e-3 / (rep + 1), 1 - b1 ** (rep + 1), 1 - b2 ** (rep + 1), 0.5], device="cuda"))
        ref = kept(step(d, eager, scalars))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(out, ref, f"replay {rep}")
        for a, b in zip(state(par), state(eager)):
            assert torch.equal(a, b), f"replay {rep}: weights or states"


def test_graphs_of_one_input_do_not_share_memory():
    """Two captured steps over the same inputs, replayed in turn: nothing of one is in the other."""
    d, one, two = inputs(5), parameters(6), parameters(7)
    step(d, parameters(6))
    graphs, outs = [], []
    for par in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(d, par, update=False))
        graphs.append(g)
    refs = [kept(step(d, q, update=False)) for q in (parameters(6), parameters(7))]
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        same(outs[i], refs[i], f"graph {i}")


def test_side_stream_argument():
    d, par = inputs(8), parameters(9)
    ref = kept(step(d, parameters(9)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        par = parameters(9)
        torch.cuda.synchronize()
        got = step(d, par, stream=stream)
        torch.cuda.synchronize()
        same(got, ref, f"stream {stream}")


def test_two_threads():
    refs = [kept(step(inputs(20 + i), parameters(30 + i))) for i in range(2)]
    torch.cuda.synchronize()
    results, errors = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                d = inputs(20 + i)
                for _ in range(5):
                    got = step(d, parameters(30 + i))
                results[i] = kept(got)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        same(results[i], refs[i], f"thread {i}")


def test_outputs_stay_inside_their_buffers():
    d = inputs(11)
    tr = fq.fp8q_moe_sort(d["ids"], d["x"], E0, LOCAL)[2]
    off, trg, rt, xs = (Guarded((LOCAL + 1,), torch.int32), Guarded((T, K_TOP), torch.int32), Guarded((CAP,), torch.int32),
                        Guarded((CAP, H), torch.bfloat16))
    for n in (T, 1):    # several routing chunks' worth of entries and the single launch
        run("fp8q_moe_sort", p(d["ids"]), n, K_TOP, E0, LOCAL, p(d["x"]), fq.FP8Q_OUT_BF16, H, n * K_TOP, xs.ptr, off.ptr,
            trg.ptr, rt.ptr)
        assert_intact(off, trg, rt, xs)
    dx, dw = Guarded((T, H), torch.float32), Guarded((T, K_TOP), torch.float32)
    run("fp8q_moe_sort_backward", p(xs.t), fq.FP8Q_OUT_BF16, CAP, H, p(tr), T, K_TOP, dx.ptr, fq.FP8Q_OUT_F32)
    dout = Guarded((CAP, H), torch.bfloat16)
    run("fp8q_moe_combine_backward", p(d["dy"]), fq.FP8Q_OUT_BF16, p(xs.t), fq.FP8Q_OUT_BF16, CAP, H, p(tr), p(d["gate"]), T,
        K_TOP, dout.ptr, dw.ptr)
    assert_intact(dx, dw, dout)
    M, inner = 77, 264
    gu, dh = torch.randn((M, 2 * inner), device="cuda").bfloat16(), torch.randn((M, inner), device="cuda")
    dgu, h = Guarded((M, 2 * inner), torch.bfloat16), Guarded((M, inner), torch.bfloat16)
    run("fp8q_swiglu_backward", p(gu), p(dh), fq.FP8Q_OUT_F32, M, inner, dgu.ptr, h.ptr)
    assert_intact(dgu, h)
    # a division of the rows that uses every tile there can be: one row in each expert but the last
    G, M, K = 5, 4 + 128, 256
    offs = torch.tensor([0, 1, 2, 3, 4, M], dtype=torch.int32, device="cuda")
    x = torch.randn((M, K), device="cuda").bfloat16()
    tiles = M // 128 + G
    for rows in (True, False):
        xq, sa = Guarded((M, K), torch.uint8), Guarded((K // 128, M), torch.float32)
        xt, st = Guarded((tiles, K, 128), torch.uint8), Guarded((tiles, K), torch.float32)
        run("fp8q_quantize_act_grouped", p(x), p(offs), G, M, K, xq.ptr if rows else None, sa.ptr if rows else None, xt.ptr,
            st.ptr)
        assert_intact(xq, sa, xt, st)
    for dtype, code in ((torch.float32, fq.FP8Q_OUT_F32), (torch.bfloat16, fq.FP8Q_OUT_BF16)):
        c = Guarded((G, K, K), dtype)
        run("fp8q_grouped_gemm_rowscaled", p(xt.t), p(st.t), p(xt.t), p(st.t), p(offs), G, M, K, K, c.ptr, code)
        assert_intact(c)


def test_invalid_offsets_stay_inside():
    """Offsets that no routing gives (decreasing, negative, overlapping, far too large): results are
    unspecified, but nothing outside the buffers is touched."""
    G, M, K = 6, 300, 128
    x = torch.randn((M, K), device="cuda").bfloat16()
    tiles = M // 128 + G
    top = 2 ** 31 - 1
    for offs in ([0, 300, 0, 300, 0, 300, 0], [-5, -1, 400, 200, top, -top, 300], [0, top, 0, top, 0, top, 0], [300] * 7):
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        xq, sa = Guarded((M, K), torch.uint8), Guarded((K // 128, M), torch.float32)
        xt, st = Guarded((tiles, K, 128), torch.uint8), Guarded((tiles, K), torch.float32)
        xt.t.zero_(), st.t.zero_()
        run("fp8q_quantize_act_grouped", p(x), p(o), G, M, K, xq.ptr, sa.ptr, xt.ptr, st.ptr)
        run("fp8q_quantize_act_grouped", p(x), p(o), G, M, K, None, None, xt.ptr, st.ptr)
        c = Guarded((G, K, K), torch.float32)
        run("fp8q_grouped_gemm_rowscaled", p(xt.t), p(st.t), p(xt.t), p(st.t), p(o), G, M, K, K, c.ptr, fq.FP8Q_OUT_F32)
        assert_intact(xq, sa, xt, st, c)


def test_shared_memory_and_devices_are_refused():
    n = torch.zeros(256, device="cuda")
    z = [torch.zeros(128, device="cuda") for _ in range(3)]
    with pytest.raises(ValueError, match="share memory"):
        fq.fp8q_adamw_plan([n[:128], n[64:192]], [z[0]] * 2, [z[1], z[2]], [torch.zeros_like(z[0]) for _ in range(2)])
    with pytest.raises(ValueError, match="16-byte"):
        fq.fp8q_adamw_plan([n[1:129]], [z[0]], [z[1]], [z[2]])
    with pytest.raises(ValueError, match="128 elements"):
        fq.fp8q_adamw_plan([z[0]], [z[1]], [z[2]], [n])
    with pytest.raises(ValueError, match="shape"):
        fq.fp8q_adamw(fq.fp8q_adamw_plan([z[0]], [z[1]], [z[2]], [n[:128]]), lr=1e-3, scalars=n[:3])
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_adamw(fq.fp8q_adamw_plan([z[0]], [z[1]], [z[2]], [n[:128]]), lr=1e-3, step=0)
    with pytest.raises(ValueError):
        fq.fp8q_moe_sort(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.zeros((4, 16), device="cuda")[:, ::2], 0, 2)


# ------------------------------------------------------------------ offsets past 31 bits
def test_large_sort_and_its_gradient():
    T, k, E, H = 40960, 8, 64, 7168                        # 327680 rows x 7168: 2.3e9 elements
    g = gen(1)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    xs, off, tr, rt = fq.fp8q_moe_sort(ids, x, 0, E)
    rows = torch.tensor([0, 1, T * k // 2, T * k - 2, T * k - 1], device="cuda")
    assert torch.equal(xs[rows], x[rt[rows].long()]) and int(off[-1]) == T * k
    dx = fq.fp8q_moe_sort_backward(xs, tr, out_dtype=torch.float32)
    t = torch.tensor([0, T - 1], device="cuda")
    # k equal rows: k x, exactly (at most three more bits than BF16 holds)
    assert torch.equal(dx[t], k * x[t].float())
    w = torch.full((T, k), 0.5, device="cuda")
    dout, dw = fq.fp8q_moe_combine_backward(x, xs, tr, w)
    assert torch.equal(dout[rows], (0.5 * x[rt[rows].long()].float()).bfloat16())
    ref = x[t].double().square().sum(1)
    assert bool(((dw[t].double() - ref[:, None]).abs() <= (8 * 14 + 6) * 2.0 ** -24 * ref[:, None]).all())


def test_large_swiglu_gradient():
    M, inner = 300_000, 4096                                # 2.4e9 elements of gu
    gu = torch.zeros((M, 2 * inner), dtype=torch.bfloat16, device="cuda")
    dh = torch.ones((M, inner), dtype=torch.bfloat16, device="cuda")
    gu[-2:] = torch.randn((2, 2 * inner), device="cuda", generator=gen(2)).bfloat16()
    dgu, h = fq.fp8q_swiglu_backward(gu, dh, want_h=True)
    small = fq.fp8q_swiglu_backward(gu[-2:].clone(), dh[-2:].clone(), want_h=True)
    assert torch.equal(dgu[-2:], small[0]) and torch.equal(h[-2:], small[1]) and not bool(dgu[0].any())


def test_large_token_tiles_and_product():
    M, P, Q, G = 300_032, 7168, 128, 3                        # 2.15e9 codes
    off = torch.tensor([0, 150_000, 299_900, M], dtype=torch.int32, device="cuda")
    dy = torch.randn((M, P), device="cuda", generator=gen(3)).bfloat16()
    x = torch.randn((M, Q), device="cuda", generator=gen(4)).bfloat16()
    a, sa = fq.fp8q_quantize_act_grouped(dy, off, rows=False)[2:]
    b, sb = fq.fp8q_quantize_act_grouped(x, off, rows=False)[2:]
    got = fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, off, M, out_dtype=torch.float32)
    last = torch.tensor([0, M - 299_900], dtype=torch.int32, device="cuda")
    n = M - 299_900
    c, sc = fq.fp8q_quantize_act_grouped(dy[-n:].clone(), last, rows=False)[2:]
    d, sd = fq.fp8q_quantize_act_grouped(x[-n:].clone(), last, rows=False)[2:]
    assert torch.equal(fq.fp8q_grouped_gemm_rowscaled(c, sc, d, sd, last, n, out_dtype=torch.float32)[0], got[2])


def test_large_adamw():
    n = 2 ** 31 + 129
    p_, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 128), device="cuda") for _ in range(2))
    g[-3:] = 1.0
    fq.fp8q_adamw(fq.fp8q_adamw_plan([p_], [g], [m], [v], [ms], [vs]), lr=0.5)
    torch.cuda.synchronize()
    assert bool(((p_[-3:] + 0.5).abs() < 1e-6).all()) and not bool(p_[:-3].any())
    assert m[-3:].tolist() == v[-3:].tolist() == [126] * 3 and not bool(m[:-3].any())   # the largest finite code
