"""The operators of a training step of an MoE layer, each in its plain form (elementary torch
operations in FP32) and as the calls of this package: tokens sorted by expert and back with
their gradients, the SwiGLU gradient, the experts' weight gradient in E4M3, and AdamW over
many tensors with states in FP32 or in E4M3.

A case holds the sizes; `prepare` makes its inputs on the GPU from a seed, `run` is one pass.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
BETAS, EPS, DECAY, LR, STEP = (0.9, 0.95), 1e-8, 0.1, 2e-4, 100


# --------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------
def listed():
    return [
        # a few tokens on a GPU that holds all 256 experts: launches and latency count
        {"name": "sort_64_tokens", "op": "sort", "T": 64, "k": 8, "experts": 256, "local": 256, "H": 7168, "dtype": "bf16",
         "short": False},
        # one training batch on a GPU with 32 of the 256 experts
        {"name": "sort_8192_tokens", "op": "sort", "T": 8192, "k": 8, "experts": 256, "local": 32, "H": 7168, "dtype": "bf16",
         "short": False},
        # a small FP32 gradient of odd sizes
        {"name": "sort_grad_ragged", "op": "sort_grad", "T": 777, "k": 4, "experts": 64, "local": 24, "H": 1000, "dtype": "f32",
         "out": "f32"},
        # the token gradient of the training batch
        {"name": "sort_grad_8192_tokens", "op": "sort_grad", "T": 8192, "k": 8, "experts": 256, "local": 32, "H": 7168,
         "dtype": "bf16", "out": "bf16"},
        # a few tokens, FP32 expert outputs, every expert local
        {"name": "combine_grad_ragged", "op": "combine_grad", "T": 301, "k": 2, "experts": 16, "local": 16, "N": 264,
         "dtype": "f32", "dy": "bf16"},
        # the training batch, every expert local: the most rows per token
        {"name": "combine_grad_8192_tokens", "op": "combine_grad", "T": 8192, "k": 8, "experts": 256, "local": 256, "N": 7168,
         "dtype": "bf16", "dy": "bf16"},
        # one small expert's rows
        {"name": "swiglu_grad_ragged", "op": "swiglu_grad", "M": 333, "I": 264, "dh": "f32", "h": False},
        # the training batch's rows on 32 experts, with h recomputed for the down projection's weight gradient
        {"name": "swiglu_grad_8192_rows", "op": "swiglu_grad", "M": 8192, "I": 2048, "dh": "bf16", "h": True},
        # up projection of 32 experts, about 256 rows each: the FP32 gradient's bytes count
        {"name": "wgrad_up_32_experts", "op": "wgrad", "G": 32, "M": 8192, "N": 4096, "K": 7168, "out": "f32", "empty": 0},
        # down projection of 4 experts that saw the tokens of many GPUs: the product counts
        {"name": "wgrad_down_4_experts", "op": "wgrad", "G": 4, "M": 16384, "N": 7168, "K": 2048, "out": "bf16", "empty": 0},
        # the many small tensors of a layer (norms, gates, biases, a small projection)
        {"name": "adamw_f32_64_tensors", "op": "adamw", "tensors": 64, "largest": 300_001, "state": "f32", "grad": "f32",
         "copy": False, "equal": False},
        # 32 experts' down projections of 7168 x 2048 with E4M3 states, BF16 gradients and the BF16 weights written too
        {"name": "adamw_e4m3_32_experts", "op": "adamw", "tensors": 32, "largest": 7168 * 2048, "state": "e4m3", "grad": "bf16",
         "copy": True, "equal": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "sort_grad", "combine_grad", "swiglu_grad", "wgrad", "adamw"])
    if op in ("sort", "sort_grad", "combine_grad"):
        experts = _spread(rng, 4, 256)
        local = experts if rng.random() < 0.4 else _spread(rng, 1, experts)
        case = {"op": op, "T": _spread(rng, 1, 8192), "k": rng.randint(1, min(8, experts)), "experts": experts, "local": local}
        width = 8 * _spread(rng, 1, 896)
        if op == "sort":
            return {**case, "H": width, "dtype": rng.choice(["bf16", "f32"]), "short": rng.random() < 0.2}
        if op == "sort_grad":
            return {**case, "H": width, "dtype": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"])}
        return {**case, "N": width, "dtype": rng.choice(["bf16", "f32"]), "dy": rng.choice(["bf16", "f32"])}
    if op == "swiglu_grad":
        return {"op": op, "M": _spread(rng, 1, 8192), "I": 8 * _spread(rng, 1, 256), "dh": rng.choice(["bf16", "f32"]),
                "h": rng.random() < 0.5}
    if op == "wgrad":
        G = _spread(rng, 1, 32)
        return {"op": op, "G": G, "M": _spread(rng, 1, 8192), "N": 128 * _spread(rng, 1, 32), "K": 128 * _spread(rng, 1, 32),
                "out": rng.choice(["bf16", "f32"]), "empty": rng.randint(0, G // 4)}
    return {"op": op, "tensors": _spread(rng, 1, 200), "largest": _spread(rng, 64, 2_000_000), "state": rng.choice(["f32", "e4m3"]),
            "grad": rng.choice(["bf16", "f32"]), "copy": rng.random() < 0.5, "equal": False}


# --------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------
def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=gen) * scale).to(DTYPES[dtype])


def _routing(gen, case):
    """Top-k of random scores with a standing preference per expert: ids [T, k] int32 and gating
    weights [T, k] that sum to one."""
    T, k, experts = case["T"], case["k"], case["experts"]
    score = torch.rand((T, experts), device="cuda", generator=gen) + 0.3 * torch.rand((1, experts), device="cuda", generator=gen)
    top = torch.topk(score, k, dim=1)
    return top.indices.to(torch.int32), (top.values / top.values.sum(1, keepdim=True)).float()


def _shares(case, seed):
    """Rows of each expert (uneven, `empty` of them with none), summing to M."""
    r = np.random.RandomState(seed % (1 << 31))
    G, M = case["G"], case["M"]
    p = np.exp(0.3 * r.standard_normal(G))
    p[r.permutation(G)[:case["empty"]]] = 0.0
    return r.multinomial(M, p / p.sum())


def _sizes(case):
    """Sizes of the tensors of an AdamW step: equal expert weights, or the spread of a layer's tensors."""
    n, top = case["tensors"], case["largest"]
    if case["equal"]:
        return [top] * n
    return [max(1, int(top ** (1 - 0.6 * i / n)) - 3 * (i % 5)) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("sort", "sort_grad", "combine_grad"):
        T, k, local = case["T"], case["k"], case["local"]
        s["ids"], s["w"] = _routing(gen, case)
        cap = max(1, T * k // 3) if case.get("short") else T * k
        if op == "sort":
            s["x"] = _normal(gen, (T, case["H"]), case["dtype"])
            s["xs"] = torch.zeros((cap, case["H"]), device="cuda", dtype=DTYPES[case["dtype"]])
            s["row_token"] = torch.zeros(cap, device="cuda", dtype=torch.int32)
            return s
        _, s["token_row"], s["row_entry"], s["n"] = _route(s["ids"], local, cap)
        if op == "sort_grad":
            s["dxs"] = _normal(gen, (cap, case["H"]), case["dtype"])
        else:
            s["out"] = _normal(gen, (cap, case["N"]), case["dtype"])
            s["dy"] = _normal(gen, (T, case["N"]), case["dy"])
            s["dout"] = torch.zeros((cap, case["N"]), device="cuda", dtype=DTYPES[case["dtype"]])
    elif op == "swiglu_grad":
        s["gu"] = _normal(gen, (case["M"], 2 * case["I"]), "bf16", 2.0)
        s["dh"] = _normal(gen, (case["M"], case["I"]), case["dh"])
    elif op == "wgrad":
        rows = _shares(case, seed)
        s["longest"] = -(-int(rows.max()) // 128) * 128
        s["offsets"] = torch.tensor([0, *np.cumsum(rows).tolist()], dtype=torch.int32, device="cuda")
        s["dy"] = _normal(gen, (case["M"], case["N"]), "bf16", 1e-3)
        s["x"] = _normal(gen, (case["M"], case["K"]), "bf16")
    else:
        sizes = _sizes(case)
        first = np.concatenate([[0], np.cumsum([-(-n // 128) * 128 for n in sizes])]).tolist()
        s["flat"] = flat = {"p": torch.zeros(first[-1], device="cuda")}
        g = torch.zeros(first[-1], device="cuda", dtype=DTYPES[case["grad"]])
        if case["copy"]:
            flat["copies"] = torch.zeros(first[-1], device="cuda", dtype=torch.bfloat16)
        m, root = torch.zeros_like(flat["p"]), torch.zeros_like(flat["p"])  # root: sqrt(v)
        for i, n in enumerate(sizes):  # the rest of each tensor's last 128 stays zero
            at = slice(first[i], first[i] + n)
            flat["p"][at].normal_(0, 0.02, generator=gen)
            g[at].normal_(0, 1e-2, generator=gen)
            m[at].normal_(0, 1e-3, generator=gen)
            root[at].uniform_(0, 1e-2, generator=gen)
        if case["state"] == "f32":
            flat["m"], flat["v"] = m, root * root
        else:
            flat["m"], flat["m_scale"] = _to_e4m3(m)
            flat["v"], flat["v_scale"] = _to_e4m3(root)
        for name, x in [*flat.items(), ("g", g)]:
            step = 128 if name.endswith("scale") else 1
            s[name] = [x[f // step:f // step + -(-n // step)] for f, n in zip(first, sizes)]
        if own:
            s["plan"] = _plan(s)
    return s


# --------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------
def _route(ids, local, cap):
    """offsets [local + 1], token_row [T, k], row_entry [cap] (the (token, slot) entry of a row) and
    the number of rows (on the device) of the entries routed to experts 0 .. local - 1."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where(flat < local, flat, local)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(n, device=ids.device))
    offsets = (key.view(-1, 1) < torch.arange(local + 1, device=ids.device)).sum(0).int()
    token_row = torch.where((key < local) & (place < cap), place, -1).int().view(ids.shape)
    return offsets, token_row, order[:cap], offsets[local].clamp(max=cap)


def _sort(s):
    case = s["case"]
    offsets, token_row, entry, n = _route(s["ids"], case["local"], s["xs"].shape[0])
    token = entry // case["k"]
    here = torch.arange(token.numel(), device=token.device) < n
    return {"xs": torch.where(here[:, None], s["x"][token], s["xs"]), "offsets": offsets, "token_row": token_row,
            "row_token": torch.where(here, token.int(), s["row_token"])}


def _rows(rows, token_row):
    """FP32 rows [T, k, H] of the slots that have one, zeros for the others."""
    return torch.where(token_row[..., None] >= 0, rows[token_row.clamp(min=0).long()].float(), 0.0)


def _sort_grad(s):
    return {"dx": _rows(s["dxs"], s["token_row"]).sum(1).to(DTYPES[s["case"]["out"]])}


def _combine_grad(s):
    case = s["case"]
    dy, entry = s["dy"].float(), s["row_entry"]
    dw = (_rows(s["out"], s["token_row"]) * dy[:, None, :]).sum(-1)
    rows = (s["w"].reshape(-1)[entry][:, None] * dy[entry // case["k"]]).to(s["dout"].dtype)
    here = torch.arange(entry.numel(), device=entry.device) < s["n"]
    return {"dout": torch.where(here[:, None], rows, s["dout"]), "dw": dw}


def _swiglu_grad(s):
    case = s["case"]
    g, u = s["gu"].float().split(case["I"], dim=1)
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    dgu = torch.cat([dh * u * (sig + silu * (1.0 - sig)), dh * silu], dim=1).bfloat16()
    return {"dgu": dgu, "h": (silu * u).bfloat16()} if case["h"] else {"dgu": dgu}


def _divided(x, s):
    """x / s, and x itself where the group is all zeros."""
    return torch.where(s > 0, x / torch.where(s > 0, s, 1.0), x)


def _over_448(amax):
    return amax / torch.full_like(amax, E4M3_MAX)  # a tensor divisor: a true division


def _to_e4m3(x):
    """E4M3 codes of a vector with an FP32 scale per 128 values."""
    n = x.numel()
    tiles = torch.nn.functional.pad(x, (0, -n % 128)).view(-1, 128)
    scale = _over_448(tiles.abs().amax(1))
    return _divided(tiles, scale[:, None]).to(torch.float8_e4m3fn).reshape(-1)[:n].view(torch.uint8).clone(), scale


def _of_e4m3(codes, scale):
    n = codes.numel()
    tiles = torch.nn.functional.pad(codes.view(torch.float8_e4m3fn).float(), (0, -n % 128)).view(-1, 128)
    return (tiles * scale[:, None]).reshape(-1)[:n]


def _token_tiles(x, offsets, longest):
    """x [M, C] by expert, quantized and back: [G, longest, C] in FP32, tiles of 128 consecutive
    tokens of one expert and one channel, the end of an expert's last tile zero."""
    first, end = offsets[:-1].long()[:, None], offsets[1:].long()[:, None]
    row = first + torch.arange(longest, device=x.device)
    there = row < end
    rows = torch.where(there[..., None], x[torch.where(there, row, 0)].float(), 0.0)
    tiles = rows.view(rows.shape[0], longest // 128, 128, x.shape[1])
    scale = _over_448(tiles.abs().amax(2, keepdim=True))
    return (_divided(tiles, scale).to(torch.float8_e4m3fn).float() * scale).view(rows.shape)


def _wgrad(s):
    a = _token_tiles(s["dy"], s["offsets"], s["longest"])
    b = _token_tiles(s["x"], s["offsets"], s["longest"])
    return {"dw": torch.bmm(a.transpose(1, 2).contiguous(), b).to(DTYPES[s["case"]["out"]])}


def _adamw_one(p, g, m, v):
    """New (p, m, v) of one tensor, FP32."""
    b1, b2 = BETAS
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * (1.0 - b2)) * g
    denominator = torch.sqrt(v) * (1.0 / math.sqrt(1.0 - b2 ** STEP)) + EPS
    return p * (1.0 - LR * DECAY) - (m / denominator) * (LR / (1.0 - b1 ** STEP)), m, v


def _adamw_f32(s, i):
    p, m, v = _adamw_one(s["p"][i], s["g"][i].float(), s["m"][i], s["v"][i])
    s["p"][i].copy_(p), s["m"][i].copy_(m), s["v"][i].copy_(v)
    return s["copies"][i].copy_(p) if "copies" in s else None


def _adamw_e4m3(s, i):
    root = _of_e4m3(s["v"][i], s["v_scale"][i])
    p, m, v = _adamw_one(s["p"][i], s["g"][i].float(), _of_e4m3(s["m"][i], s["m_scale"][i]), root * root)
    codes, scale = _to_e4m3(m)
    s["p"][i].copy_(p), s["m"][i].copy_(codes), s["m_scale"][i].copy_(scale)
    root = torch.sqrt(v)
    codes, scale = _to_e4m3(root)
    s["v"][i].copy_(torch.where((root > 0) & (codes == 0), 1, codes)), s["v_scale"][i].copy_(scale)  # no v becomes zero
    return s["copies"][i].copy_(p) if "copies" in s else None


def _adamw_outputs(s):
    """The updated tensors, end to end as they lie; E4M3 codes as values of their type."""
    return {k: x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x for k, x in s["flat"].items()}


def _adamw(s):
    one = _adamw_f32 if s["case"]["state"] == "f32" else _adamw_e4m3
    [one(s, i) for i in range(len(s["p"]))]
    return _adamw_outputs(s)


PLAIN = {"sort": _sort, "sort_grad": _sort_grad, "combine_grad": _combine_grad, "swiglu_grad": _swiglu_grad, "wgrad": _wgrad,
         "adamw": _adamw}


# --------------------------------------------------------------------------------------
# The calls of the package
# --------------------------------------------------------------------------------------
def _plan(s):
    import fp8_fine_grained_fp8q_amd as fq

    return fq.fp8q_adamw_plan(s["p"], s["g"], s["m"], s["v"], s.get("m_scale"), s.get("v_scale"), s.get("copies"))


def _run_own(s):
    import fp8_fine_grained_fp8q_amd as fq

    case = s["case"]
    op = case["op"]
    if op == "sort":
        xs, offsets, token_row, row_token = fq.fp8q_moe_sort(s["ids"], s["x"], 0, case["local"], xs=s["xs"], row_token=s["row_token"])
        return {"xs": xs, "offsets": offsets, "token_row": token_row, "row_token": row_token}
    if op == "sort_grad":
        return {"dx": fq.fp8q_moe_sort_backward(s["dxs"], s["token_row"], out_dtype=DTYPES[case["out"]])}
    if op == "combine_grad":
        dout, dw = fq.fp8q_moe_combine_backward(s["dy"], s["out"], s["token_row"], s["w"], dout=s["dout"])
        return {"dout": dout, "dw": dw}
    if op == "swiglu_grad":
        dgu, h = fq.fp8q_swiglu_backward(s["gu"], s["dh"], want_h=case["h"])
        return {"dgu": dgu, "h": h} if case["h"] else {"dgu": dgu}
    if op == "wgrad":
        _, _, a, sa = fq.fp8q_quantize_act_grouped(s["dy"], s["offsets"], rows=False)
        _, _, b, sb = fq.fp8q_quantize_act_grouped(s["x"], s["offsets"], rows=False)
        return {"dw": fq.fp8q_grouped_gemm_rowscaled(a, sa, b, sb, s["offsets"], case["M"], out_dtype=DTYPES[case["out"]])}
    fq.fp8q_adamw(s["plan"], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, step=STEP)
    return _adamw_outputs(s)


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# --------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = lambda d: 4 if d == "f32" else 2  # noqa: E731
    if op in ("sort", "sort_grad", "combine_grad"):
        T, k = case["T"], case["k"]
        rows = T * k * case["local"] / case["experts"]  # routed rows, on the whole
        seen = T * (1 - (1 - case["local"] / case["experts"]) ** k)  # tokens with one
        if op == "sort":
            rows = min(rows, T * k // 3) if case["short"] else rows
            return {"bytes": (seen + rows) * case["H"] * size(case["dtype"]) + 8 * T * k + 4 * rows, "flops": 0}
        if op == "sort_grad":
            return {"bytes": case["H"] * (rows * size(case["dtype"]) + T * size(case["out"])) + 4 * T * k, "flops": rows * case["H"]}
        return {"bytes": case["N"] * (2 * rows * size(case["dtype"]) + seen * size(case["dy"])) + 12 * T * k,
                "flops": 3 * rows * case["N"]}
    if op == "swiglu_grad":
        n = case["M"] * case["I"]
        return {"bytes": n * (8 + size(case["dh"]) + (2 if case["h"] else 0)), "flops": 10 * n}
    if op == "wgrad":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * (N + K) + case["G"] * N * K * size(case["out"]), "flops": 2 * M * N * K}
    n = sum(_sizes(case))
    state = 16 if case["state"] == "f32" else 4 + 16 / 128
    return {"bytes": n * (8 + size(case["grad"]) + state + (2 if case["copy"] else 0)), "flops": 14 * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        return _exact_sort(s)
    if op in ("sort_grad", "combine_grad"):
        at, k = s["token_row"].cpu().numpy().astype(np.int64), case["k"]
        wide = torch.zeros((at.shape[0], case["H"] if op == "sort_grad" else case["N"]), dtype=torch.float64, device="cuda")
        if op == "sort_grad":
            for j in range(k):
                t = np.nonzero(at[:, j] >= 0)[0]
                wide[t] += s["dxs"][at[t, j]].double()
            return {"dx": wide}
        dy, dout, dw = s["dy"].double(), s["dout"].double(), torch.zeros(at.shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = np.nonzero(at[:, j] >= 0)[0]
            dw[t, j] = (s["out"][at[t, j]].double() * dy[t]).sum(1)
            dout[at[t, j]] = dy[t] * s["w"][t, j].double()[:, None]
        return {"dout": dout, "dw": dw}
    if op == "swiglu_grad":
        g, u = s["gu"][:, :case["I"]].double(), s["gu"][:, case["I"]:].double()
        dh, sig = s["dh"].double(), torch.sigmoid(s["gu"][:, :case["I"]].double())
        got = {"dgu": torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)}
        return {**got, "h": g * sig * u} if case["h"] else got
    if op == "wgrad":
        ends, dw = s["offsets"].tolist(), []
        for a, b in zip(ends, ends[1:]):
            n = [torch.zeros((0, c), dtype=torch.float64, device="cuda") for c in (case["N"], case["K"])]
            for lo in range(a, b, 128):
                n = [torch.cat([x, _exact_tile(y[lo:min(lo + 128, b)])]) for x, y in zip(n, (s["dy"], s["x"]))]
            dw.append(n[0].t() @ n[1])
        return {"dw": torch.stack(dw)}
    return _exact_adamw(s)


def _exact_sort(s):
    ids, local, cap = s["ids"].cpu().numpy(), s["case"]["local"], s["xs"].shape[0]
    xs = s["xs"].double()
    where = [np.nonzero(ids.reshape(-1) == e)[0] for e in range(local)]
    entries = np.concatenate(where)[:cap] // s["case"]["k"]
    xs[:len(entries)] = s["x"][entries].double()
    return {"xs": xs}


def _exact_tile(x):
    """A tile of at most 128 tokens as its codes and scales stand for it. The scale and the quotient are
    FP32 by definition, and E4M3 has 4 significant bits down to 2^-6, then steps of 2^-9."""
    x = x.double()
    scale = (x.abs().amax(0) / 448).float().double()
    y = torch.where(scale > 0, x / scale, x).float().double()
    step = torch.exp2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return torch.round(y / step) * step * scale


def _exact_adamw(s):
    case, (b1, b2) = s["case"], BETAS
    new = {k: x.double() for k, x in s["flat"].items() if k in ("p", "copies")}
    f32 = case["state"] == "f32"
    if f32:
        new |= {k: s["flat"][k].double() for k in ("m", "v")}
    at = 0
    for i, p in enumerate(s["p"]):
        n, p, g = p.numel(), p.double(), s["g"][i].double()
        if f32:
            m, v = s["m"][i].double(), s["v"][i].double()
        else:
            spread = torch.arange(n, device="cuda") // 128
            m, v = (s[k][i].view(torch.float8_e4m3fn).double() * s[k + "_scale"][i].double()[spread] for k in ("m", "v"))
            v = v.square()
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g.square()
        p = p - LR * (DECAY * p + m / (1 - b1 ** STEP) / ((v / (1 - b2 ** STEP)).sqrt() + EPS))
        for k, x in (("p", p), ("copies", p), ("m", m), ("v", v)):
            if k in new:
                new[k][at:at + n] = x
        at += -(-n // 128) * 128
    return new
