"""GPU parity of the MoE layer's backward pieces against plain references in 64 bits.

* fp8q_moe_sort: rows, offsets and maps equal to the oracle's dispatch of the same ids.
* fp8q_moe_sort_backward, fp8q_moe_combine_backward, fp8q_swiglu_backward: within the bound of
  their FP32 operations and of the output's rounding (half a step: BF16 2^-8, FP32 2^-24
  relative), and the formulas of the gradients against differences of the forward oracle.
* fp8q_quantize_act_grouped: codes and scales bit-exact against the oracle's quantizers applied
  to each expert's rows filled up with zeros.
* fp8q_grouped_gemm_rowscaled: within 2e-3 ||a_row|| ||b_row|| of the oracle's FP64 product (and
  the rounding of the output), and with FP32 output within the bound of FP32 sums.
Rows and columns that belong to nobody keep the sentinel they held before the call."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq
import workloads as wl
from oracle import backward as ob
from oracle import gemm as og
from oracle import moe as om
from oracle import quant as oq

from helpers import assert_quant_equal, dev, dev_bf16, host

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative
TYPES = [torch.bfloat16, torch.float32]


def values(shape, dtype, seed, scale=1.0):
    """Seeded device values and the same in float64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)
    return t, t.double().cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, tol, what):
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    err = np.abs(got - ref)
    bad = err > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance, worst err/tol {np.max(err / np.maximum(tol, 1e-300)):.3g}"
    print(f"[{what}] max err/tol {float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0:.3f}", flush=True)


# ------------------------------------------------------------------ sort, and its gradient
# one wave's chunk and several, k = 1 and 64, one expert and 1024, nothing local, short capacity; one
# routing chunk, a few that count for themselves, and more that share the counts
SORTS = [(1, 1, 1, 0, 8, 1, None), (300, 8, 20, 16, 264, 64, None), (77, 1, 5, 0, 2056, 64, None),
         (40, 64, 128, 0, 8, 128, None), (700, 8, 1024, 0, 24, 1500, None), (64, 6, 1, 9, 128, 8, None),
         (200, 4, 16, 0, 4104, 16, 333), (50, 2, 8, 0, 64, 8, 0),
         (2100, 8, 1024, 0, 8, 1024, None), (2200, 8, 64, 0, 16, 80, None), (2200, 8, 64, 0, 16, 1, 9000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,e_begin,H,ids,cap", SORTS)
def test_sort(T, k, E, e_begin, H, ids, cap, dtype):
    rng = np.random.default_rng(T + k + E + H)
    idx = rng.integers(0, ids, size=(T, k)).astype(np.int32)     # duplicates and other GPUs' experts included
    x, _ = values((T, H), dtype, T)
    cap = T * k if cap is None else cap
    xs = torch.full((cap, H), -7.0, dtype=dtype, device="cuda")
    rt = torch.full((cap,), -9, dtype=torch.int32, device="cuda")
    out = fq.fp8q_moe_sort(dev(idx), x, e_begin, E, xs=xs, row_token=rt)
    torch.cuda.synchronize()
    roff, rrt, rtr = om.dispatch(idx, e_begin, E)
    n = min(int(roff[-1]), cap)
    assert out[0] is xs and np.array_equal(host(out[1]), roff)
    assert np.array_equal(host(out[2]), np.where(rtr < cap, rtr, -1))
    assert np.array_equal(host(rt)[:n], rrt[:n]) and np.all(host(rt)[n:] == -9)
    assert torch.equal(xs[:n], x[dev(rrt[:n])]) and bool((xs[n:] == -7.0).all())


def test_sort_without_tokens():
    off = fq.fp8q_moe_sort(torch.empty((0, 8), dtype=torch.int32, device="cuda"),
                           torch.empty((0, 64), dtype=torch.float32, device="cuda"), 0, 5)[1]
    torch.cuda.synchronize()
    assert host(off).tolist() == [0] * 6


def test_sort_matches_dispatch_maps():
    """The two ways of routing the same ids agree, and the sorted values quantize to the
    dispatched codes."""
    ids, _ = wl.topk_routing(seed=5, tokens=700, experts=64, topk=4)
    x, _ = values((700, 384), torch.bfloat16, 3)
    xq, sa = fq.fp8q_quantize_act_1x128(x)
    xs, ss, off, tr, rt = fq.fp8q_moe_dispatch(dev(ids), xq, sa, 8, 24)
    vs, off2, tr2, rt2 = fq.fp8q_moe_sort(dev(ids), x, 8, 24)
    vq, vsa = fq.fp8q_quantize_act_1x128(vs)
    n = int(off[-1])
    assert n > 0 and torch.equal(off, off2) and torch.equal(tr, tr2) and torch.equal(rt[:n], rt2[:n])
    assert torch.equal(vq[:n], xs[:n]) and torch.equal(vsa[:, :n], ss[:, :n])


def maps(T, k, experts, local, seed, cap=None):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, size=(T, k)).astype(np.int32)
    _, _, tr = om.dispatch(ids, 0, local)
    cap = T * k if cap is None else cap
    return np.where(tr < cap, tr, -1).astype(np.int32), cap


# the token without a row, every slot with one, k = 64, several workgroups per token, a short capacity
MAPS = [(1, 1, 1, 1, 8, None), (300, 8, 64, 8, 264, None), (33, 64, 70, 70, 16, None), (65, 3, 8, 8, 4104, None),
        (129, 4, 16, 16, 1000, 200), (20, 2, 900, 1, 72, None)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("T,k,experts,local,H,cap", MAPS)
def test_sort_backward(T, k, experts, local, H, cap, dtype, out_dtype):
    tr, cap = maps(T, k, experts, local, T + H, cap)
    dxs, ref_dxs = values((cap, H), dtype, H)
    used = np.zeros(cap, bool)
    used[tr[tr >= 0]] = True
    dxs[torch.from_numpy(~used).cuda()] = float("nan")            # rows of nobody are not read
    got = f64(fq.fp8q_moe_sort_backward(dxs, dev(tr), out_dtype=out_dtype))
    one = np.ones(tr.shape)
    ref = om.combine(ref_dxs, tr, one)
    # k - 1 FP32 additions, then the rounding of the output
    tol = (k - 1) * 2.0 ** -24 * om.combine_bound(ref_dxs, tr, one) * (1 + 2.0 ** -8) + HALF[out_dtype] * np.abs(ref)
    within(got, ref, tol, f"sort_backward {T} {k} {H}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dy_dtype", TYPES)
@pytest.mark.parametrize("T,k,experts,local,N,cap", MAPS)
def test_combine_backward(T, k, experts, local, N, cap, dtype, dy_dtype):
    tr, cap = maps(T, k, experts, local, T + N, cap)
    out, ref_out = values((cap, N), dtype, N)
    dy, ref_dy = values((T, N), dy_dtype, N + 1)
    w = np.random.default_rng(N).random((T, k)).astype(np.float32)
    w[0, 0] = 0.0
    used = np.zeros(cap, bool)
    used[tr[tr >= 0]] = True
    out[torch.from_numpy(~used).cuda()] = float("nan")
    dout = torch.full((cap, N), -7.0, dtype=dtype, device="cuda")
    got, dw = fq.fp8q_moe_combine_backward(dy, out, dev(tr), dev(w), dout=dout)
    torch.cuda.synchronize()
    t, s = np.nonzero(tr >= 0)
    r = tr[t, s]
    ref = w.astype(np.float64)[t, s, None] * ref_dy[t]
    # an FP32 product, then the rounding of the output
    within(f64(got)[r], ref, (2.0 ** -24 * (1 + 2.0 ** -7) + HALF[dtype]) * np.abs(ref), f"dout {T} {k} {N}")
    assert bool((got[torch.from_numpy(~used).cuda()] == -7.0).all())
    ref_dw = np.zeros((T, k))
    ref_dw[t, s] = (ref_out[r] * ref_dy[t]).sum(1)
    bound = np.zeros((T, k))
    bound[t, s] = np.abs(ref_out[r] * ref_dy[t]).sum(1)
    # a lane adds up to 8 ceil(N / 512) products, then 6 additions join the lanes
    depth = 8 * -(-N // 512) + 6
    within(f64(dw), ref_dw, depth * 2.0 ** -24 * (1 + 1e-3) * bound, f"dw {T} {k} {N}")


def test_combine_gradients_against_differences():
    """The gradients' formulas: central differences of L = <dy, combine(out, w)> (float64 oracle)."""
    T, k, N = 12, 3, 16
    tr, cap = maps(T, k, 6, 4, 7)
    out, o64 = values((cap, N), torch.float32, 1)
    dy, d64 = values((T, N), torch.float32, 2)
    w = np.random.default_rng(3).random((T, k)).astype(np.float32)
    dout, dw = fq.fp8q_moe_combine_backward(dy, out, dev(tr), dev(w), dout=torch.zeros_like(out))
    w64 = w.astype(np.float64)

    def loss(o, ww):
        return float((d64 * om.combine(o, tr, ww)).sum())

    for r, c in [(0, 0), (1, 5), (int(tr.max()), N - 1)]:
        e = np.zeros_like(o64)
        e[r, c] = 0.5
        assert abs(loss(o64 + e, w64) - loss(o64 - e, w64) - f64(dout)[r, c]) < 1e-5
    for t in range(T):
        for s in range(k):
            e = np.zeros_like(w64)
            e[t, s] = 0.5
            assert abs(loss(o64, w64 + e) - loss(o64, w64 - e) - f64(dw)[t, s]) < 1e-4


# ------------------------------------------------------------------ SwiGLU gradient
def swiglu_refs(gu, dh):
    I = dh.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    t = np.exp(-np.abs(g))
    s = np.where(g >= 0, 1.0, t) / (1.0 + t)
    c = np.where(g >= 0, t, 1.0) / (1.0 + t)
    return g, u, s, c, np.concatenate([dh * u * s * (1 + g * c), dh * g * s], 1), g * u * s


@pytest.mark.parametrize("dh_dtype", TYPES)
@pytest.mark.parametrize("M,I", [(1, 8), (3, 264), (333, 128), (7, 2048), (1000, 40)])
@pytest.mark.parametrize("scale", [1.0, 20.0])
def test_swiglu_backward(M, I, scale, dh_dtype):
    gu, gu64 = values((M, 2 * I), torch.bfloat16, M + I, scale)
    gu[0, :4] = torch.tensor([0.0, -100.0, 100.0, -1.2784645], dtype=torch.bfloat16)   # 0, both ends, dg's zero
    gu64 = f64(gu)
    dh, dh64 = values((M, I), dh_dtype, M * 3 + I)
    dgu, h = fq.fp8q_swiglu_backward(gu, dh, want_h=True)
    torch.cuda.synchronize()
    g, u, s, c, ref, ref_h = swiglu_refs(gu64, dh64)
    # e^-|g| and the reciprocal 2 half-steps each, 1 + t, the products and the FMA one each: at
    # most 16 half-steps of the largest term; then the rounding to BF16 (and its subnormals)
    big = np.concatenate([np.abs(dh64 * u) * s * (1 + np.abs(g) * c), np.abs(dh64 * g) * s], 1)
    within(f64(dgu), ref, 16 * 2.0 ** -24 * big * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 1e-38, f"dgu {M} {I}")
    within(f64(h), ref_h, (16 * 2.0 ** -24 * (1 + 2.0 ** -8) + 2.0 ** -8) * np.abs(ref_h) + 1e-38, f"h {M} {I}")
    again, none = fq.fp8q_swiglu_backward(gu, dh)
    assert none is None and torch.equal(again, dgu)


def test_swiglu_backward_against_differences():
    gu, gu64 = values((4, 32), torch.bfloat16, 5, 2.0)
    dh, dh64 = values((4, 16), torch.float32, 6)
    dgu = f64(fq.fp8q_swiglu_backward(gu, dh)[0])
    eps = 1e-5
    for r in range(4):
        for col in range(32):
            e = np.zeros_like(gu64)
            e[r, col] = eps
            up, down = (np.sum(dh64 * swiglu_refs(gu64 + x, dh64)[5]) for x in (e, -e))
            # the difference's own error is of the order of eps^2; the output is BF16
            assert abs((up - down) / (2 * eps) - dgu[r, col]) < 2.0 ** -8 * abs(dgu[r, col]) + 1e-6


# ------------------------------------------------------------------ token tiles per expert
# empty experts (first, middle, last), 1, 127, 128, 129 rows, more than 64 experts
COUNTS = [[1], [128], [0, 0, 0], [129, 0, 127], [0, 300, 1, 0], [5] * 70, [0] * 64 + [130] + [0] * 9 + [2]]


def grouped_reference(x, counts):
    """Oracle codes [tiles][K][128] and scales [tiles][K] of the experts' tiles in order."""
    q, s, at, K = [np.zeros((0, x.shape[1], 128), np.uint8)], [np.zeros((0, x.shape[1]), np.float32)], 0, x.shape[1]
    for n in counts:
        for lo in range(0, n, 128):
            tile = np.zeros((128, K), np.uint16)
            tile[:min(128, n - lo)] = x[at + lo:at + min(lo + 128, n)]
            a, b = ob.quantize_act_128x1(tile)
            q.append(a[None]), s.append(b)
        at += n
    return np.concatenate(q), np.concatenate(s)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("slack", [0, 37])
@pytest.mark.parametrize("counts", COUNTS)
def test_quantize_act_grouped(counts, slack):
    K, n = 256, sum(counts)
    M, G = n + slack, len(counts)
    rng = np.random.default_rng(M + G)
    x = wl.bf16_bits((rng.standard_normal((M, K)) * np.logspace(-2, 2, K)).astype(np.float32))
    if n > 5:
        x[:n, 7] = 0                                             # an all-zero channel
        x[2, 9] = wl.bf16_bits(np.array([5e4], np.float32))[0]
    tiles = M // 128 + G
    bufs = [torch.full(shape, 0xA5 if d == torch.uint8 else -3.0, dtype=d, device="cuda")
            for shape, d in (((M, K), torch.uint8), ((K // 128, M), torch.float32), ((tiles, K, 128), torch.uint8),
                             ((tiles, K), torch.float32))]
    off = dev(offsets_of(counts))
    xq, sa, xqt, sat = fq.fp8q_quantize_act_grouped(dev_bf16(x), off, xq=bufs[0], sa=bufs[1], xqt=bufs[2], sat=bufs[3])
    torch.cuda.synchronize()
    rq, rs = grouped_reference(x, counts)
    w = rq.shape[0]
    assert w <= tiles
    assert_quant_equal(xqt[:w], sat[:w], rq, rs, "token tiles")
    assert bool((xqt[w:] == 0xA5).all()) and bool((sat[w:] == -3.0).all())
    fwd, fsa = oq.quantize_act_1x128(x[:n]) if n else (np.zeros((0, K), np.uint8), np.zeros((K // 128, 0), np.float32))
    assert_quant_equal(xq[:n].contiguous(), sa[:, :n].contiguous(), fwd, fsa, "rows")
    assert bool((xq[n:] == 0xA5).all()) and bool((sa[:, n:] == -3.0).all())
    none, none2, only, onlys = fq.fp8q_quantize_act_grouped(dev_bf16(x), off, rows=False)
    assert none is None and none2 is None
    assert torch.equal(only[:w], xqt[:w]) and torch.equal(onlys[:w], sat[:w])


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("counts,P,Q,slack", [([1], 128, 128, 0), ([129, 0, 700], 384, 256, 0), ([0, 0], 128, 256, 0),
                                              ([40] * 66, 128, 128, 5), ([1030, 5], 640, 896, 300),
                                              ([0, 2500], 256, 512, 0)])
def test_grouped_weight_gradient(counts, P, Q, slack, out_dtype):
    n, G = sum(counts), len(counts)
    M = n + slack
    dy, _ = values((M, P), torch.bfloat16, M + P, 1e-3)
    x, _ = values((M, Q), torch.bfloat16, M + Q)
    off = dev(offsets_of(counts))
    a, sa = fq.fp8q_quantize_act_grouped(dy, off, rows=False)[2:]
    b, sb = fq.fp8q_quantize_act_grouped(x, off, rows=False)[2:]
    w = sum(-(-c // 128) for c in counts)
    # what lies behind the tiles must not reach the product: NaN codes and scales
    a[w:], b[w:], sa[w:], sb[w:] = 0x7F, 0x7F, float("nan"), float("nan")
    got = fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, off, M, out_dtype=out_dtype)
    torch.cuda.synchronize()
    at = 0
    for g, c in enumerate(counts):
        tiles = slice(at, at + -(-c // 128))
        at = tiles.stop
        if c == 0:
            assert bool((got[g] == 0).all())
            continue
        # the tiles side by side are the operands of the dense product
        h = [host(t[tiles]) for t in (a, sa, b, sb)]
        h[0], h[2] = (np.ascontiguousarray(q.transpose(1, 0, 2).reshape(q.shape[1], -1)) for q in (h[0], h[2]))
        ref = ob.wgrad(*h)
        # the acceptance bound is on the accumulation; with one token |C| = ||a|| ||b||, and
        # BF16's half step of 2^-8 |C| alone is above 2e-3 ||a|| ||b||, so it is added
        tol = og.tolerance(ob.row_norms_rowscaled(h[0], h[1]), ob.row_norms_rowscaled(h[2], h[3]))
        if out_dtype == torch.float32:
            # 128 additions in a tile, two scalings, one addition per tile
            total = np.abs(oq.dequant_act(h[0], h[1])) @ np.abs(oq.dequant_act(h[2], h[3])).T
            tol = np.minimum(tol, (130 + -(-c // 128)) * 2.0 ** -24 * (1 + 1e-4) * total)
        within(f64(got[g]), ref, tol + HALF[out_dtype] * np.abs(ref), f"expert {g}")


@pytest.mark.parametrize("out_dtype", TYPES)
def test_runs_of_tiles(out_dtype):
    """Many experts with few tokens, where a workgroup takes several tiles in a row (the last run
    of a row shorter): the same bits as each expert alone, tile by tile."""
    counts = [100, 0, 200, 300, 1, 128, 129, 31, 257, 33] * 4
    G, P, Q, M = len(counts), 1280, 1408, sum(counts)
    dy, _ = values((M, P), torch.bfloat16, 1, 1e-3)
    x, _ = values((M, Q), torch.bfloat16, 2)
    off = dev(offsets_of(counts))
    a, sa = fq.fp8q_quantize_act_grouped(dy, off, rows=False)[2:]
    b, sb = fq.fp8q_quantize_act_grouped(x, off, rows=False)[2:]
    got = fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, off, M, out_dtype=out_dtype)
    at = 0
    for g, c in enumerate(counts):
        one = dev(offsets_of([c]))
        ops = [fq.fp8q_quantize_act_grouped(t[at:at + c].contiguous(), one, rows=False)[2:] for t in (dy, x)]
        at += c
        assert torch.equal(fq.fp8q_grouped_gemm_rowscaled(*ops[0], *ops[1], one, c, out_dtype=out_dtype)[0], got[g]), g


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("counts,P,Q,slack", [([1500, 900], 8320, 512, 0),
                                              ([1, 0, 129, 259, 385, 64, 4000, 5000], 384, 2048, 7),
                                              ([0, 0, 5120, 0], 512, 4096, 100), ([2900, 900], 8320, 512, 0),
                                              ([1, 0, 129, 259, 385, 64, 6000, 8000], 384, 2048, 7),
                                              ([0, 0, 7000, 0], 512, 4096, 100)])
def test_wide_tiles(counts, P, Q, slack, out_dtype):
    """Gradients of experts with many tokens, computed in tiles of 256 x 128 (the last one of a P
    of 128 modulo 256 half empty): experts without tokens and of one to 40 token tiles, the same
    bits as each expert alone in the small tiles, rows and tokens behind them not touched."""
    G, M = len(counts), sum(counts) + slack
    dy, _ = values((M, P), torch.bfloat16, 3, 1e-3)
    x, _ = values((M, Q), torch.bfloat16, 4)
    off = dev(offsets_of(counts))
    a, sa = fq.fp8q_quantize_act_grouped(dy, off, rows=False)[2:]
    b, sb = fq.fp8q_quantize_act_grouped(x, off, rows=False)[2:]
    w = sum(-(-c // 128) for c in counts)
    a[w:], b[w:], sa[w:], sb[w:] = 0x7F, 0x7F, float("nan"), float("nan")
    all_c = torch.full((G + 2, P, Q), 7.0, dtype=out_dtype, device="cuda")
    got = fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, off, M, out=all_c[1:G + 1])
    torch.cuda.synchronize()
    assert bool((all_c[0] == 7.0).all()) and bool((all_c[-1] == 7.0).all())
    rows = list(range(0, 40)) + list(range(P - 150, P - 110)) + list(range(P - 20, P))
    at = row = 0
    for g, c in enumerate(counts):
        tiles = slice(at, at + -(-c // 128))
        at, row = tiles.stop, row + c
        if c == 0:
            assert bool((got[g] == 0).all())
            continue
        one = dev(offsets_of([c]))
        ops = [fq.fp8q_quantize_act_grouped(t[row - c:row].contiguous(), one, rows=False)[2:] for t in (dy, x)]
        assert torch.equal(fq.fp8q_grouped_gemm_rowscaled(*ops[0], *ops[1], one, c, out_dtype=out_dtype)[0], got[g]), g
        h = [host(t) for t in (a[tiles][:, rows], sa[tiles][:, rows], b[tiles], sb[tiles])]
        h[0], h[2] = (np.ascontiguousarray(q.transpose(1, 0, 2).reshape(q.shape[1], -1)) for q in (h[0], h[2]))
        ref = ob.wgrad(*h)
        tol = og.tolerance(ob.row_norms_rowscaled(h[0], h[1]), ob.row_norms_rowscaled(h[2], h[3]))
        if out_dtype == torch.float32:
            # 128 additions in a tile, two scalings, one addition per tile
            total = np.abs(oq.dequant_act(h[0], h[1])) @ np.abs(oq.dequant_act(h[2], h[3])).T
            tol = np.minimum(tol, (130 + -(-c // 128)) * 2.0 ** -24 * (1 + 1e-4) * total)
        within(f64(got[g][rows]), ref, tol + HALF[out_dtype] * np.abs(ref), f"expert {g}")


def test_grouped_weight_gradient_without_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    ops = [torch.zeros((3, 128, 128), dtype=torch.uint8, device="cuda"), torch.zeros((3, 128), device="cuda")] * 2
    got = fq.fp8q_grouped_gemm_rowscaled(*ops, off, 0, out=torch.full((3, 128, 128), 5.0, device="cuda"))
    torch.cuda.synchronize()
    assert bool((got == 0).all())


def test_short_capacity_clamps_both_alike():
    """Offsets that count more rows than there are (a capacity too small): the quantizer and the
    product clamp them alike."""
    counts, M = [100, 200, 300], 250
    off = dev(offsets_of(counts))
    kept = [100, 150, 0]
    dy, _ = values((M, 128), torch.bfloat16, 1)
    x, _ = values((M, 256), torch.bfloat16, 2)
    res = []
    for o in (off, dev(offsets_of(kept))):
        a, sa = fq.fp8q_quantize_act_grouped(dy, o, rows=False)[2:]
        b, sb = fq.fp8q_quantize_act_grouped(x, o, rows=False)[2:]
        res.append(fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, o, M, out_dtype=torch.float32))
    assert torch.equal(res[0], res[1])
