"""The grouped weight gradient with scales from all over FP32: products of two scales past its largest
number and below its normal ones, where the gradient itself is finite and normal.  Tokens of
one operand against other tokens of the other give 0, not inf * 0; one smallest code against one
smallest code gives what it is; and a gradient of small scales keeps FP32's accuracy."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_fp8q_amd as fq

from helpers import dev

pytestmark = pytest.mark.gpu

ACCEPT = 2e-3   # the products' acceptance bound, here of the sum of the terms' magnitudes


def operand(tiles, C, seed):
    """Codes of magnitude 64 to 416 with random signs, scales between 1/4 and 4."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0x68, 0x7E, (tiles, C, 128), device="cuda", generator=g, dtype=torch.uint8)
    q |= torch.randint(0, 2, q.shape, device="cuda", generator=g, dtype=torch.uint8) << 7
    return q, torch.exp2(4 * torch.rand((tiles, C), device="cuda", generator=g) - 2)


def extremes(q, s, at, firsts, other):
    """Channels at .. at + 24 and what they hold in the experts' first tiles and in every tile."""
    a, b, c = slice(at, at + 8), slice(at + 8, at + 16), slice(at + 16, at + 24)
    s[firsts, a] *= 2.0 ** (70 if other else 80)         # with the other's: 2^150, but no token of both
    q[firsts, a] = torch.where((torch.arange(128, device="cuda") >= 64) == other, q[firsts, a], 0)
    q[firsts, a, 0] = 0
    s[:, b] *= 2.0 ** (-43 if other else -100)           # 2^-143
    q[firsts, c] = 0
    q[firsts, c, 0] = 1                                  # 2^-9 each
    s[firsts, c] = 2.0 ** (60 if other else 70)          # 2^130 * 2^-18


# small tiles alone, in runs of several with more columns than runs, and wide ones
SIZES = [([300, 0, 1, 129], 256, 384), ([60, 0, 200, 128] * 10, 1920, 2176), ([1700, 1500, 1601, 1699], 4096, 2048),
         ([1700, 1500, 1601, 1699], 3968, 2176)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,P,Q", SIZES)
def test_scales_of_any_size(counts, P, Q, out_dtype):
    G, M = len(counts), sum(counts)
    off = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    tiles = M // 128 + G
    used = [-(-n // 128) for n in counts]
    first = np.concatenate([[0], np.cumsum(used)]).tolist()
    firsts = [first[g] for g in range(G) if used[g]]
    (a, sa), (b, sb) = operand(tiles, P, 1), operand(tiles, Q, 2)
    for at in (0, P - 128):
        extremes(a, sa, at, firsts, False)
    for at in (0, Q - 128):
        extremes(b, sb, at, firsts, True)
    for g, n in enumerate(counts):                        # no tokens behind an expert's last one
        if n % 128:
            a[first[g + 1] - 1, :, n % 128:] = 0
            b[first[g + 1] - 1, :, n % 128:] = 0
    got = fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, off, M, out_dtype=out_dtype)
    half = 2.0 ** (-8 if out_dtype == torch.bfloat16 else -24)
    for g in range(G):
        ref, total = (torch.zeros((P, Q), dtype=torch.float64, device="cuda") for _ in range(2))
        for t in range(first[g], first[g + 1]):
            x, y = (q[t].view(torch.float8_e4m3fn).double() * s[t].double()[:, None] for q, s in ((a, sa), (b, sb)))
            ref += x @ y.t()
            total += x.abs() @ y.abs().t()
        out = got[g].double()
        assert not bool(out.isnan().any()), f"expert {g}: {int(out.isnan().sum())} NaN"
        # FP32: 128 additions in a tile, two scalings, one addition per tile; BF16 output: the bound of
        # its matrix instructions; then the rounding of the output, and what FP32's subnormals lose
        # in each tile's two scalings and addition
        sums = (130 + used[g]) * 2.0 ** -24 * (1 + 1e-4) if out_dtype == torch.float32 else ACCEPT
        tol = sums * total + half * ref.abs() + (3 * used[g] + 1) * 2.0 ** -149 + (2.0 ** -134 if half > 2.0 ** -24 else 0)
        over = ref.abs() - tol > 3.4e38
        assert bool(torch.isinf(out[over]).all())
        err = (out - ref).abs()[~over] - tol[~over]
        assert bool((err <= 0).all()), f"expert {g}: {int((err > 0).sum())} of {err.numel()} out of tolerance"


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,P,Q", SIZES)
def test_scales_far_from_one_with_ordinary_products(counts, P, Q, out_dtype):
    """One operand 2^70 times larger, the other as much smaller, and channels of zeros: the products of the
    scales are what they were, and so is every bit of the gradient."""
    G, M = len(counts), sum(counts)
    off = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    tiles = M // 128 + G
    (a, sa), (b, sb) = operand(tiles, P, 3), operand(tiles, Q, 4)
    for q, s, at in ((a, sa, P // 3), (b, sb, Q // 2)):
        q[:, at], s[:, at] = 0, 0
        q[0, at + 1], s[0, at + 1] = 0, 0
    got = [fq.fp8q_grouped_gemm_rowscaled(a, sa * x, b, sb / x, off, M, out_dtype=out_dtype) for x in (1.0, 2.0 ** 70, 2.0 ** -75)]
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    assert not bool(got[0][:, P // 3].any()) and not bool(got[0][:, :, Q // 2].any())
