"""The operators around the experts in a training step of an MoE layer, each in its plain form
(elementary torch operations in FP32) and as the calls of this package: the norm before the router,
the router's top-k with the balance loss, their gradients, and Muon, the optimizer whose update of a
weight matrix is made orthogonal by Newton-Schulz products.

A case holds the sizes; `prepare` makes its inputs on the GPU from a seed, `run` is one pass.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5  # of a norm
ALPHA, SCALE = 1e-3, 2.5  # of the balance loss, of the gating weights
A, B, C = COEFFICIENTS = (3.4445, -4.7750, 2.0315)  # of a Newton-Schulz step, x' = (A + B x x^T + C (x x^T)^2) x
STEPS = 5
LR, BETA, DECAY = 1e-4, 0.95, 0.1


# --------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------
def listed():
    return [
        # the tokens of a small decoding batch, RMS norm: the call itself counts
        {"name": "norm_64_tokens", "op": "norm", "T": 64, "H": 7168, "center": False, "x": "bf16", "out": "bf16"},
        # a training batch, layer norm of FP32 residuals into the BF16 that the quantizers read
        {"name": "norm_16384_tokens", "op": "norm", "T": 16384, "H": 7168, "center": True, "x": "f32", "out": "bf16"},
        # a small FP32 layer of odd sizes
        {"name": "norm_grad_ragged", "op": "norm_grad", "T": 777, "H": 1000, "center": True, "x": "f32", "dy": "f32", "out": "f32"},
        # the training batch's gradient, with the sums over all of its tokens for weight and bias
        {"name": "norm_grad_8192_tokens", "op": "norm_grad", "T": 8192, "H": 7168, "center": True, "x": "bf16", "dy": "bf16",
         "out": "bf16"},
        # the tokens of a small decoding batch over 256 experts, sigmoid scores and a selection bias
        {"name": "route_64_tokens", "op": "route", "B": 1, "S": 64, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "normalize": True, "logits": "f32", "padded": False},
        # four padded sequences, each with its own balance loss
        {"name": "route_16384_tokens", "op": "route", "B": 4, "S": 4096, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "normalize": True, "logits": "f32", "padded": True},
        # a small router of odd sizes with plain softmax probabilities as weights
        {"name": "route_grad_ragged", "op": "route_grad", "B": 3, "S": 111, "E": 60, "k": 3, "score": "softmax", "bias": False,
         "normalize": False, "logits": "bf16", "padded": True},
        # the gradient for the four sequences
        {"name": "route_grad_16384_tokens", "op": "route_grad", "B": 4, "S": 4096, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "normalize": True, "logits": "f32", "padded": True},
        # a small matrix of odd sizes
        {"name": "orthogonalize_300x1000", "op": "orthogonalize", "G": 1, "P": 300, "Q": 1000, "x": "f32"},
        # the weight matrix of a dense layer
        {"name": "orthogonalize_4096x7168", "op": "orthogonalize", "G": 1, "P": 4096, "Q": 7168, "x": "bf16"},
        # the router's own weight matrix
        {"name": "muon_256x7168", "op": "muon", "G": 1, "P": 256, "Q": 7168, "grad": "f32", "nesterov": True, "copy": False},
        # 32 experts' down projections, the BF16 weights for the quantizer written too
        {"name": "muon_32_experts", "op": "muon", "G": 32, "P": 7168, "Q": 2048, "grad": "bf16", "nesterov": True, "copy": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "route", "route_grad", "orthogonalize", "muon"])
    pick = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op in ("norm", "norm_grad"):
        case = {"op": op, "T": _spread(rng, 1, 8192), "H": 8 * _spread(rng, 1, 1024), "center": rng.random() < 0.6, "x": pick(), "out": pick()}
        return case if op == "norm" else {**case, "dy": pick()}
    if op in ("route", "route_grad"):
        E, B = _spread(rng, 4, 512), _spread(rng, 1, 8)
        return {"op": op, "B": B, "S": _spread(rng, 1, 8192 // B), "E": E, "k": rng.randint(1, min(8, E)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "normalize": rng.random() < 0.6,
                "logits": pick(), "padded": rng.random() < 0.5}
    P, Q = _spread(rng, 8, 2048), _spread(rng, 8, 2048)
    if op == "orthogonalize":
        return {"op": op, "G": _spread(rng, 1, 4), "P": P, "Q": Q, "x": pick()}
    return {"op": op, "G": _spread(rng, 1, 16), "P": P, "Q": Q, "grad": pick(), "nesterov": rng.random() < 0.7,
            "copy": rng.random() < 0.5}


# --------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------
def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=gen) * scale).to(DTYPES[dtype])


def _activations(gen, T, H, dtype):
    """Tokens with channels of their own mean, and one channel in 500 far larger than the others."""
    x = torch.randn((T, H), device="cuda", generator=gen) + 0.3 * torch.randn((1, H), device="cuda", generator=gen)
    far = torch.rand((1, H), device="cuda", generator=gen) < 0.002
    return torch.where(far, 30.0 * x, x).to(DTYPES[dtype])


def _gradient(gen, case, dtype):
    """Matrices as gradients are: a few strong directions over a floor of noise."""
    G, P, Q = case["G"], case["P"], case["Q"]
    r = min(16, P, Q)
    strong = torch.randn((G, P, r), device="cuda", generator=gen) * (0.7 ** torch.arange(r, device="cuda"))
    x = torch.bmm(strong, torch.randn((G, r, Q), device="cuda", generator=gen))
    return ((x + 0.5 * torch.randn((G, P, Q), device="cuda", generator=gen)) * 1e-3).to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        s["x"] = _activations(gen, T, H, case["x"])
        s["weight"] = 1.0 + _normal(gen, (H,), "f32", 0.1)
        s["bias"] = _normal(gen, (H,), "f32", 0.1) if case["center"] else None
        if op == "norm_grad":
            s["dy"] = _normal(gen, (T, H), case["dy"], 1e-3)
            x = s["x"].float()  # what the forward pass has kept
            mean = x.mean(1) if case["center"] else None
            x = x - mean[:, None] if case["center"] else x
            s["mean"], s["rstd"] = mean, 1.0 / torch.sqrt((x * x).mean(1) + EPS)
    elif op in ("route", "route_grad"):
        n, S, E = case["B"], case["S"], case["E"]
        logits = torch.randn((n, S, E), device="cuda", generator=gen) + 0.5 * torch.randn((1, 1, E), device="cuda", generator=gen)
        s["logits"] = logits.to(DTYPES[case["logits"]])
        s["bias"] = _normal(gen, (E,), "f32", 0.02) if case["bias"] else None
        s["valid"] = None
        if case["padded"]:
            long = (torch.rand((n, 1), device="cuda", generator=gen) * 0.7 + 0.3) * S
            s["valid"] = torch.arange(S, device="cuda") < long
        if op == "route_grad":
            ids, w, _, _, slope = _route(s).values()
            s["ids"], s["w"], s["slope"] = ids.contiguous(), w.contiguous(), slope
            s["dw"] = _normal(gen, (n, S, case["k"]), "f32", 1e-3)
            s["dloss"] = torch.ones(1, device="cuda")
    elif op == "orthogonalize":
        s["x"] = _gradient(gen, case, case["x"])
    else:
        shape = (case["G"], case["P"], case["Q"])
        s["grad"] = _gradient(gen, case, case["grad"])
        s["momentum"] = 3.0 * _gradient(gen, case, "f32") + s["grad"].float()
        s["param"] = _normal(gen, shape, "f32", 0.02)
        s["copy"] = torch.zeros(shape, device="cuda", dtype=torch.bfloat16) if case["copy"] else None
    return s


# --------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------
def _norm(s):
    case, x = s["case"], s["x"].float()
    mean = x.mean(1) if case["center"] else None
    x = x - mean[:, None] if case["center"] else x
    rstd = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
    y = x * rstd[:, None] * s["weight"]
    y = (y + s["bias"] if case["center"] else y).to(DTYPES[case["out"]])
    return {"y": y, "mean": mean, "rstd": rstd} if case["center"] else {"y": y, "rstd": rstd}


def _norm_grad(s):
    case, x, dy = s["case"], s["x"].float(), s["dy"].float()
    x = (x - s["mean"][:, None] if case["center"] else x) * s["rstd"][:, None]
    g = dy * s["weight"]
    dx = g - x * (g * x).mean(1, keepdim=True)
    dx = dx - g.mean(1, keepdim=True) if case["center"] else dx
    got = {"dx": (dx * s["rstd"][:, None]).to(DTYPES[case["out"]]), "dweight": (dy * x).sum(0)}
    return {**got, "dbias": dy.sum(0)} if case["center"] else got


def _sigmoid(z):
    t = torch.exp(-z.abs())
    return torch.where(z >= 0, 1.0, t) / (1.0 + t)


def _softmax(z):
    t = torch.exp(z - z.amax(-1, keepdim=True))
    return t / t.sum(-1, keepdim=True)


def _route(s):
    case, z = s["case"], s["logits"].float()
    soft, k, E = case["score"] == "softmax", case["k"], case["E"]
    score = _softmax(z) if soft else _sigmoid(z)
    rank = z  # either score rises with the logit
    if case["bias"]:  # near ties: ranked in 64 bits
        rank = (_softmax(z.double()) if soft else _sigmoid(z.double())) + s["bias"].double()
    ids = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :k]  # ties: the lowest index
    valid = torch.ones(z.shape[:2], dtype=torch.bool, device=z.device) if s["valid"] is None else s["valid"]
    w = torch.gather(score, -1, ids)
    w = SCALE * (w / w.sum(-1, keepdim=True) if case["normalize"] else w)
    ids = torch.where(valid[..., None], ids, -1).int()
    counts = (ids.reshape(z.shape[0], -1, 1) == torch.arange(E, device=z.device)).sum(1).int()
    p = torch.where(valid[..., None], score if soft else score / score.sum(-1, keepdim=True), 0.0).sum(1)
    tokens = valid.sum(1, keepdim=True)
    routed = (counts.sum(1, keepdim=True).double() * tokens).clamp(min=1)
    slope = (ALPHA / case["B"] * E * counts.double() / routed).float()
    return {"ids": ids, "w": torch.where(valid[..., None], w, 0.0), "counts": counts, "loss": (slope * p).sum().reshape(1),
            "slope": slope}


def _route_grad(s):
    case, z = s["case"], s["logits"].float()
    soft = case["score"] == "softmax"
    valid = s["ids"][..., :1] >= 0
    score = _softmax(z) if soft else _sigmoid(z)
    p = score if soft else score / score.sum(-1, keepdim=True)
    slope = s["slope"][:, None, :] * s["dloss"]
    dz = p * (slope - (p * slope).sum(-1, keepdim=True)) * (1.0 if soft else 1.0 - score)
    ids = s["ids"].clamp(min=0).long()
    dw, w = torch.where(valid, s["dw"], 0.0), s["w"]
    if case["normalize"]:  # a softmax over the chosen ones
        d = w * (dw - (w * dw).sum(-1, keepdim=True) / SCALE)
    else:
        d = w * dw
    if not soft:
        d = d * (1.0 - torch.gather(score, -1, ids))
    dz = dz + torch.zeros_like(z).scatter_(-1, ids, d)
    if soft and not case["normalize"]:
        dz = dz - p * (w * dw).sum(-1, keepdim=True)
    return {"dlogits": torch.where(valid, dz, 0.0).to(s["logits"].dtype)}


def _newton_schulz(x):
    """x [G, P, Q] in FP32 with its singular values brought near one, in FP32."""
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    norm = torch.sqrt((x.double() * x.double()).sum((1, 2), keepdim=True)).float()
    x = x / torch.where(norm > 0, norm, 1.0)
    for _ in range(STEPS):
        a = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = A * x + torch.bmm(B * a + C * torch.bmm(a, a), x)
    return x.transpose(1, 2).contiguous() if tall else x


def _orthogonalize(s):
    return {"out": _newton_schulz(s["x"].float()).bfloat16()}


def _rms(case):
    return 0.2 * math.sqrt(max(case["P"], case["Q"]))


def _muon_outputs(s):
    got = {"param": s["param"], "momentum": s["momentum"]}
    return got if s["copy"] is None else {**got, "copy": s["copy"]}


def _muon(s):
    case, g = s["case"], s["grad"].float()
    s["momentum"].copy_(BETA * s["momentum"] + g)
    u = g + BETA * s["momentum"] if case["nesterov"] else s["momentum"]
    s["param"].copy_(s["param"] * (1.0 - LR * DECAY) - (LR * _rms(case)) * _newton_schulz(u))
    if s["copy"] is not None:
        s["copy"].copy_(s["param"])
    return _muon_outputs(s)


PLAIN = {"norm": _norm, "norm_grad": _norm_grad, "route": _route, "route_grad": _route_grad, "orthogonalize": _orthogonalize,
         "muon": _muon}


# --------------------------------------------------------------------------------------
# The calls of the package
# --------------------------------------------------------------------------------------
def _run_own(s):
    import fp8_fine_grained_fp8q_amd as fq

    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd = fq.fp8q_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, center=case["center"],
                                           out_dtype=DTYPES[case["out"]])
        return {"y": y, "mean": mean, "rstd": rstd} if case["center"] else {"y": y, "rstd": rstd}
    if op == "norm_grad":
        dx, dweight, dbias = fq.fp8q_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                                         want_bias=case["center"], out_dtype=DTYPES[case["out"]])
        return {"dx": dx, "dweight": dweight, "dbias": dbias} if case["center"] else {"dx": dx, "dweight": dweight}
    if op == "route":
        ids, w, counts, loss, slope = fq.fp8q_moe_route(s["logits"], case["k"], bias=s["bias"], valid=s["valid"],
                                                        score=case["score"], normalize=case["normalize"], scale=SCALE,
                                                        balance=ALPHA)
        return {"ids": ids, "w": w, "counts": counts, "loss": loss, "slope": slope}
    if op == "route_grad":
        return {"dlogits": fq.fp8q_moe_route_backward(s["logits"], s["ids"], s["w"], s["dw"], s["slope"], s["dloss"],
                                                      score=case["score"], normalize=case["normalize"], scale=SCALE)}
    if op == "orthogonalize":
        return {"out": fq.fp8q_orthogonalize(s["x"], steps=STEPS, coefficients=COEFFICIENTS)}
    fq.fp8q_muon(s["param"], s["grad"], s["momentum"], lr=LR, beta=BETA, nesterov=case["nesterov"], weight_decay=DECAY,
                 scale=_rms(case), steps=STEPS, coefficients=COEFFICIENTS, copy=s["copy"])
    return _muon_outputs(s)


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# --------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = lambda d: 4 if d == "f32" else 2  # noqa: E731
    if op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        rows = size(case["x"]) + size(case["out"]) + (size(case["dy"]) if op == "norm_grad" else 0)
        side = 2 if case["center"] else 1
        return {"bytes": T * (H * rows + 4 * side) + 4 * H * (1 if op == "norm" and side == 1 else 2 if side == 1 else 3 if op == "norm_grad" else 2),
                "flops": T * H * (8 if op == "norm" else 12)}
    if op in ("route", "route_grad"):
        T, E, k = case["B"] * case["S"], case["E"], case["k"]
        logits = T * E * size(case["logits"])
        if op == "route":
            return {"bytes": logits + 8 * T * k + 8 * case["B"] * E + (T if case["padded"] else 0), "flops": 10 * T * E}
        return {"bytes": 2 * logits + 12 * T * k + 4 * case["B"] * E, "flops": 15 * T * E}
    m, n = sorted((case["P"], case["Q"]))
    G, elements = case["G"], case["G"] * case["P"] * case["Q"]
    flops = G * STEPS * (m * m * n + m * m * m + 2 * m * m * n)  # the two symmetric products by halves
    if op == "orthogonalize":
        return {"bytes": elements * (size(case["x"]) + 2), "flops": flops}
    return {"bytes": elements * (size(case["grad"]) + 16 + (2 if case["copy"] else 0)), "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s)
    if op == "route":
        return _exact_route(s)
    if op == "route_grad":
        return _exact_route_grad(s)
    if op == "orthogonalize":
        return {"out": torch.stack([_exact_orthogonal(x.double()) for x in s["x"]])}
    m = BETA * s["momentum"].double() + s["grad"].double()
    got = {"param": s["param"].double() * (1 - LR * DECAY), "momentum": m}
    for i in range(case["G"]):
        u = s["grad"][i].double() + BETA * m[i] if case["nesterov"] else m[i]
        got["param"][i] -= LR * _rms(case) * _exact_orthogonal(u)
    return got if s["copy"] is None else {**got, "copy": got["param"]}


def _exact_norm(s):
    case = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    if case["op"] == "norm":
        mean = x.mean(1) if case["center"] else torch.zeros(len(x), dtype=torch.float64, device="cuda")
        rstd = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt()
        y = (x - mean[:, None]) * (rstd[:, None] * w)
        return {"y": y + s["bias"].double(), "mean": mean, "rstd": rstd} if case["center"] else {"y": y, "rstd": rstd}
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    hat = (x - s["mean"].double()[:, None] if case["center"] else x) * rstd
    along = torch.stack([(dy * w * hat).mean(1), (dy * w).mean(1) * float(case["center"])])
    dx = rstd * (dy * w - hat * along[0][:, None] - along[1][:, None])
    got = {"dx": dx, "dweight": torch.einsum("th,th->h", dy, hat)}
    return {**got, "dbias": dy.sum(0)} if case["center"] else got


def _exact_route(s):
    case, E = s["case"], s["case"]["E"]
    z = s["logits"].double().cpu().numpy()
    valid = np.ones(z.shape[:2], dtype=bool) if s["valid"] is None else s["valid"].cpu().numpy()
    if case["score"] == "softmax":
        score = np.exp(z - z.max(-1, keepdims=True))
        score = share = score / score.sum(-1, keepdims=True)
    else:
        score = 1 / (1 + np.exp(-z))
        share = score / score.sum(-1, keepdims=True)
    rank = z if s["bias"] is None else score + s["bias"].double().cpu().numpy()
    ids = np.argsort(-rank, axis=-1, kind="stable")[..., :case["k"]]
    w = np.take_along_axis(score, ids, -1)
    w = SCALE * w / (w.sum(-1, keepdims=True) if case["normalize"] else 1.0) * valid[..., None]
    slope = np.zeros((case["B"], E))
    for b in range(case["B"]):
        count = np.bincount(ids[b][valid[b]].reshape(-1), minlength=E)
        slope[b] = ALPHA / case["B"] * E * count / max(1, count.sum()) / max(1, valid[b].sum())
    loss = sum((slope[b] * share[b][valid[b]].sum(0)).sum() for b in range(case["B"]))
    of = lambda a: torch.from_numpy(np.asarray(a))  # noqa: E731
    return {"ids": None, "w": of(w), "counts": None, "loss": of([loss]), "slope": of(slope)}


def _exact_route_grad(s):
    """From the derivative of each gating weight by each logit."""
    case = s["case"]
    z, ids = s["logits"].double(), s["ids"].long()
    keep = (ids[..., 0] >= 0).double()[..., None]
    at = torch.nn.functional.one_hot(ids.clamp(min=0), case["E"]).double()  # [B, S, k, E]
    slope, dw = s["slope"].double()[:, None, :] * s["dloss"].double(), s["dw"].double()
    if case["score"] == "softmax":
        score = share = torch.softmax(z, -1)
        by_score = lambda d: score * (d - (score * d).sum(-1, keepdim=True))  # noqa: E731
    else:
        score = torch.sigmoid(z)
        share = score / score.sum(-1, keepdim=True)
        by_score = lambda d: score * (1 - score) * d  # noqa: E731
    chosen = (at * score[..., None, :]).sum(-1)
    if case["normalize"]:
        total = chosen.sum(-1, keepdim=True)
        d = SCALE * (dw / total - (dw * chosen).sum(-1, keepdim=True) / total.square())
    else:
        d = SCALE * dw
    d = (at * d[..., None]).sum(2)
    if case["score"] == "softmax":
        d = d + slope
    else:
        d = d + (slope - (slope * share).sum(-1, keepdim=True)) / score.sum(-1, keepdim=True)
    return {"dlogits": by_score(d) * keep}


def _exact_orthogonal(x):
    """The polynomial of the singular values, by products with the smaller Gram matrix."""
    if x.shape[0] > x.shape[1]:
        return _exact_orthogonal(x.t()).t()
    x = x / torch.linalg.matrix_norm(x)
    for _ in range(STEPS):
        gram = x @ x.t()
        y = gram @ x
        x = A * x + B * y + C * (gram @ y)
    return x
