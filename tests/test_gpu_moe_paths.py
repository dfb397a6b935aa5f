"""The launches of the value sort and of the grouped weight gradient that a call takes by its size: the
sort's single launch, the routing whose chunks count for themselves, the three routing launches, short
and long rows, tails and short capacities, in full, between guard bytes, captured and replayed, and
on two threads; runs of several tiles per workgroup; and offsets that no routing gives in the
wide tiles."""
import threading

import numpy as np
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
from oracle import moe as om

from helpers import dev, host
from test_gpu_guard import Guarded, assert_intact, p, run

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


def routed(T, k, ids, seed):
    return np.random.default_rng(seed).integers(0, ids, size=(T, k)).astype(np.int32)


def values(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


# T, k, E, e_begin, H, ids, cap: up to 2047 entries one launch; up to 17407 the routing in one; beyond, in
# three.  Rows of up to 512 16-byte chunks, and longer ones with one, a ragged and three workgroups each
SORTS = [(2100, 1, 16, 0, 4104, 32, None), (600, 4, 16, 0, 9224, 24, 700), (2200, 8, 8, 0, 2056, 64, None),
         (2048, 1, 1, 0, 8, 1, 2000), (2175, 8, 40, 5, 4112, 60, None), (2176, 8, 40, 5, 12296, 60, 9001),
         (300, 64, 1024, 0, 520, 1500, None), (5000, 5, 3, 1, 20488, 200, 300)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,e_begin,H,ids,cap", SORTS)
def test_sort_in_full(T, k, E, e_begin, H, ids, cap, dtype):
    idx = routed(T, k, ids, T + H)
    x = values((T, H), dtype, T)
    cap = T * k if cap is None else cap
    roff, rrt, rtr = om.dispatch(idx, e_begin, E)
    n = min(int(roff[-1]), cap)
    xs, rt = Guarded((cap, H), dtype), Guarded((cap,), torch.int32)
    off, tr = Guarded((E + 1,), torch.int32), Guarded((T, k), torch.int32)
    xs.t.fill_(-7.0), rt.t.fill_(-9)
    ids_dev = dev(idx)
    run("fp8q_moe_sort", p(ids_dev), T, k, e_begin, E, p(x), fq._out_code(dtype), H, cap, xs.ptr, off.ptr, tr.ptr, rt.ptr)
    assert_intact(xs, rt, off, tr)
    assert np.array_equal(host(off.t), roff) and np.array_equal(host(tr.t), np.where(rtr < cap, rtr, -1))
    assert np.array_equal(host(rt.t)[:n], rrt[:n]) and bool((rt.t[n:] == -9).all())
    assert torch.equal(xs.t[:n], x[dev(rrt[:n])]) and bool((xs.t[n:] == -7.0).all())
    # the gradient over these maps: T rows of a token's rows, each of them x[t], added in order
    dx = Guarded((T, H), torch.float32)
    run("fp8q_moe_sort_backward", xs.ptr, fq._out_code(dtype), cap, H, tr.ptr, T, k, dx.ptr, fq.FP8Q_OUT_F32)
    assert_intact(dx)
    count = dev((host(tr.t) >= 0).sum(1).astype(np.int32))
    ref, err = x.double() * count[:, None], count[:, None] * 2.0 ** -24
    assert bool(((dx.t.double() - ref).abs() <= err * ref.abs()).all())


# the routing counts for itself, then in three launches; BF16 long rows, FP32 ragged ones
STEPS = [(600, 4, 24, 9224, torch.bfloat16), (2500, 8, 40, 1032, torch.float32)]


def sorted_back(d):
    xs, off, tr, rt = fq.fp8q_moe_sort(d["ids"], d["x"], 2, d["E"], xs=d["xs"], row_token=d["rt"])
    dout, dw = fq.fp8q_moe_combine_backward(d["x"], xs, tr, d["w"], dout=d["dout"])
    return [xs, off, tr, rt, dout, dw, fq.fp8q_moe_sort_backward(dout, tr, out_dtype=torch.float32)]


def state(T, k, E, H, dtype, seed):
    cap = T * k - 5
    return {"ids": dev(routed(T, k, 2 * E, seed)), "x": values((T, H), dtype, seed), "E": E,
            "w": values((T, k), torch.float32, seed + 1), "xs": torch.zeros((cap, H), dtype=dtype, device="cuda"),
            "dout": torch.zeros((cap, H), dtype=dtype, device="cuda"),
            "rt": torch.zeros(cap, dtype=torch.int32, device="cuda")}


@pytest.mark.parametrize("T,k,E,H,dtype", STEPS)
def test_captured_sort(T, k, E, H, dtype):
    d, eager = state(T, k, E, H, dtype, 1), state(T, k, E, H, dtype, 1)
    sorted_back(state(T, k, E, H, dtype, 1))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sorted_back(d)
    for rep in range(3):
        fresh = state(T, k, E, H, dtype, 10 + rep)
        for s in (d, eager):
            for name in ("ids", "x", "w"):
                s[name].copy_(fresh[name])
        ref = sorted_back(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b), f"replay {rep}"


def test_sorts_on_two_threads():
    refs = [[t.clone() for t in sorted_back(state(*s, 20))] for s in STEPS]
    torch.cuda.synchronize()
    results, errors = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                d = state(*STEPS[i], 20)
                for _ in range(5):
                    out = sorted_back(d)
                results[i] = [t.clone() for t in out]
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for got, ref in zip(results, refs):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def offsets_of(counts):
    return dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


# experts of no, one, two and three token tiles; a row of 17 tiles, so that the last run of four or two is
# shorter
RUNS = {"up to three token tiles each": ([0, 100, 128, 129, 256, 300, 384, 1] * 8, 2048, 2176),
        "about 100 tokens each": ([0, 100, 128, 129, 40, 300, 3, 1] * 8, 2048, 2176),
        "one token each": ([1, 0, 1, 2] * 20, 1920, 2176)}


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("name", RUNS)
def test_long_runs_of_tiles(name, out_dtype):
    counts, P, Q = RUNS[name]
    M, off = sum(counts), offsets_of(counts)
    dy, x = values((M, P), torch.bfloat16, 1, 1e-3), values((M, Q), torch.bfloat16, 2)
    a, sa = fq.fp8q_quantize_act_grouped(dy, off, rows=False)[2:]
    b, sb = fq.fp8q_quantize_act_grouped(x, off, rows=False)[2:]
    w = sum(-(-c // 128) for c in counts)
    a[w:], b[w:], sa[w:], sb[w:] = 0x7F, 0x7F, float("nan"), float("nan")
    got = torch.full((len(counts), P, Q), 5.0, dtype=out_dtype, device="cuda")
    for rep in range(3):
        fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, off, M, out=got)
    at = 0
    for g, c in enumerate(counts):
        if c == 0:
            assert not bool(got[g].any()), g
            continue
        one = offsets_of([c])
        ops = [fq.fp8q_quantize_act_grouped(t[at:at + c].contiguous(), one, rows=False)[2:] for t in (dy, x)]
        at += c
        assert torch.equal(fq.fp8q_grouped_gemm_rowscaled(*ops[0], *ops[1], one, c, out_dtype=out_dtype)[0], got[g]), g


@pytest.mark.parametrize("out_dtype", TYPES)
def test_invalid_offsets_in_wide_tiles(out_dtype):
    """Results are unspecified, but nothing outside the buffers is touched."""
    G, M, P, Q, top = 2, 3400, 4096, 2048, 2 ** 31 - 1
    tiles = M // 128 + G
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randint(0, 0x7E, (tiles, n, 128), device="cuda", generator=g, dtype=torch.uint8) for n in (P, Q))
    sa, sb = torch.ones((tiles, P), device="cuda"), torch.ones((tiles, Q), device="cuda")
    for offs in ([0, M, M], [0, M, 0], [M, 0, M], [-5, top, -top], [top, -top, top], [-top, top, M], [M] * 3):
        c = Guarded((G, P, Q), out_dtype)
        run("fp8q_grouped_gemm_rowscaled", p(a), p(sa), p(b), p(sb), p(torch.tensor(offs, dtype=torch.int32, device="cuda")), G, M,
            P, Q, c.ptr, fq._out_code(out_dtype))
        assert_intact(c)
