"""The grouped weight gradient of buffers with room for more rows than are routed, as the value sort's
default capacity makes them: the number of rows that counts is in the offsets, on the device.  The
kernels choose their tiles and runs by it, and the results are those of buffers that fit, bit for
bit, eagerly and where a captured call is replayed with few and with many rows."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

from helpers import dev

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


def offsets_of(counts):
    return dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


def spread(G, rows, seed):
    p = np.exp(0.5 * np.random.default_rng(seed).standard_normal(G))
    return np.random.default_rng(seed + 1).multinomial(rows, p / p.sum()).tolist()


def operands(dy, x, off, M):
    """Token tiles in buffers for M rows; NaN codes and scales where no tile is written."""
    out = []
    for t in (dy, x):
        full = torch.full((M, t.shape[1]), float("nan"), dtype=torch.bfloat16, device="cuda")
        full[:t.shape[0]] = t
        tiles = M // 128 + off.numel() - 1
        q = torch.full((tiles, t.shape[1], 128), 0x7F, dtype=torch.uint8, device="cuda")
        s = torch.full((tiles, t.shape[1]), float("nan"), device="cuda")
        out += fq.fp8q_quantize_act_grouped(full, off, rows=False, xqt=q, sat=s)[2:]
    return out


def rows_of(n, P, Q, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.randn((n, P), device="cuda", generator=g) * 1e-3).bfloat16(),
            torch.randn((n, Q), device="cuda", generator=g).bfloat16())


# G, routed rows, P, Q, rows that there is room for: wide tiles by the room, small ones by the rows, in runs
# of one and of several; both ways the wide ones, more of them than the grid; runs alone
SIZES = [(4, 300, 4096, 2048, 9000), (32, 4000, 1280, 2176, 65536), (8, 20000, 4352, 3968, 20500), (8, 20000, 4352, 3968, 80000),
         (40, 2000, 1920, 2176, 20000), (4, 0, 4096, 2048, 9000), (4, 6500, 4096, 2048, 6500)]


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("G,rows,P,Q,M", SIZES)
def test_room_for_more_rows(G, rows, P, Q, M, out_dtype):
    counts = spread(G, rows, G + rows)
    off = offsets_of(counts)
    dy, x = rows_of(rows, P, Q, 1)
    around = torch.full((G + 2, P, Q), 7.0, dtype=out_dtype, device="cuda")
    got = fq.fp8q_grouped_gemm_rowscaled(*operands(dy, x, off, M), off, M, out=around[1:G + 1])
    torch.cuda.synchronize()
    assert bool((around[0] == 7.0).all()) and bool((around[-1] == 7.0).all())
    at = 0
    for g, n in enumerate(counts):
        if n == 0:
            assert not bool(got[g].any())
            continue
        one = offsets_of([n])
        a, sa = fq.fp8q_quantize_act_grouped(dy[at:at + n].contiguous(), one, rows=False)[2:]
        b, sb = fq.fp8q_quantize_act_grouped(x[at:at + n].contiguous(), one, rows=False)[2:]
        at += n
        assert torch.equal(fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, one, n, out_dtype=out_dtype)[0], got[g]), g


@pytest.mark.parametrize("out_dtype", TYPES)
def test_replays_with_few_and_many_rows(out_dtype):
    G, P, Q, M = 4, 4096, 2048, 9000
    dy, x = rows_of(M, P, Q, 3)
    off = offsets_of(spread(G, M, 1))

    def step():
        a, sa = fq.fp8q_quantize_act_grouped(dy, off, rows=False)[2:]
        b, sb = fq.fp8q_quantize_act_grouped(x, off, rows=False)[2:]
        return fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, off, M, out_dtype=out_dtype)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i, rows in enumerate((M, 100, 8000, 0, 3000, 6143, 6144, 4095, 4096, M)):
        off.copy_(offsets_of(spread(G, rows, 10 + i)))
        ref = step().clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), rows
        assert bool(torch.isfinite(out).all()) and bool(out.any()) == (rows > 0)
